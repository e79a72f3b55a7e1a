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
// whatever the pages' scales are.  The sum of the row, the reference and O stay
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
// which keeps 2 to 4 KB a warp on the way.  (The same bytes through a ring of
// cp.async in shared memory took 466 instructions a tile instead of 3xx and half
// as long again: 434 us instead of xxx for 64 x 16000 x 8 heads.)
//
// Work.  One chunk = 16 W positions (a 16-position tile for each of the W
// warps) of one (sequence, kv head, row tile).  All chunks of a call lie in one
// line, which is cut into P equal ranges, one per resident CTA, whatever the
// sequences' lengths are; each CTA finds its range from the lengths on the
// device.  A unit (sequence, kv head, row tile) that is cut leaves partial sums
// in the workspace, joined by the last CTA of every 16 to arrive and then by
// the last of those, in a fixed order: results do not depend on the order of
// arrival.
#include <cuda_fp16.h>

#include <atomic>

#include "common.cuh"
#include "decode.h"
#include "kernels.h"

namespace w4q {

namespace {

constexpr float NEG = -1e30f;      // the reference before any position was seen
constexpr float SLACK = 8.f;       // the reference may lag this far (log2) behind the largest term
constexpr float P_SCALE = 128.f;   // 2^7: P <= 2^8 becomes at most 2^15 in f16
constexpr int JOIN = 16;           // partial sums joined by one CTA
constexpr int MAX_SEQS = 4096;

struct AttnParams {
    Kv8 c;
    const __nv_bfloat16 *q;
    int64_t q_stride;  // elements between query tokens
    __nv_bfloat16 *out;
    float *lse;
    int queries, heads, group, rows, row_tiles, window;
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
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// The chunks of a sequence: its first 16-position tile that some query sees
// and the number of chunks of W tiles from there, at least one.
struct Span {
    int len, first, chunks;
};
template <int W>
__device__ __forceinline__ Span span_of(const AttnParams &p, int b)
{
    Span s;
    const long long cap = (long long)p.c.width << p.c.page_log2;
    const long long len = p.c.lens[b];
    s.len = (int)(len < 0 ? 0 : (len > cap ? cap : len));
    const int lo = p.window > 0 ? s.len - p.queries - p.window + 1 : 0;
    s.first = lo > 0 ? lo >> 4 : 0;
    const int tiles = ((s.len + 15) >> 4) - s.first;
    s.chunks = tiles > 0 ? (tiles + W - 1) / W : 1;
    return s;
}

// Dynamic shared memory of a CTA: the warps' sums, then the chunks' prefix
// sums over the sequences.
template <int D, int NT, int W>
struct Smem {
    static constexpr int ROWS = 8 * NT;
    static constexpr int PITCH = D + 4;           // rows 2t, 2t + 1 of a half-warp fall into other banks
    static constexpr int BASE = ((W * ROWS * PITCH + 2 * W * ROWS) * 4 + 15) / 16 * 16;
    static size_t bytes(int seqs) { return BASE + (size_t)(seqs + 1) * 4; }
};

template <int D, int NT, bool FP8, int W, int CPS>
__global__ void __launch_bounds__(32 * W, CPS) kv8_attention_kernel(const AttnParams p)
{
    using SM = Smem<D, NT, W>;
    constexpr int ROWS = SM::ROWS, THREADS = 32 * W, KC = D / 64, VB = D / 8, VW = VB / 4, NM = D / 16;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ unsigned s_last;
    __shared__ int s_warp[W];
    float *s_o = reinterpret_cast<float *>(smem);             // [W][ROWS][PITCH]
    float *s_m = s_o + W * ROWS * SM::PITCH;                  // [W][ROWS]
    float *s_l = s_m + W * ROWS;                              // [W][ROWS]
    int *s_prefix = reinterpret_cast<int *>(smem + SM::BASE); // [seqs + 1] chunks before a sequence

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;

    pdl_wait();
    pdl_launch_dependents();

    // --- prefix sums of the sequences' chunks
    {
        int base = 0;
        for (int b0 = 0; b0 < p.c.seqs; b0 += THREADS) {
            const int b = b0 + tid;
            const int n = b < p.c.seqs ? span_of<W>(p, b).chunks : 0;
            int x = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(~0u, x, o);
                if (lane >= o)
                    x += y;
            }
            if (lane == 31)
                s_warp[warp] = x;
            __syncthreads();
            int before = base, all = base;
#pragma unroll
            for (int w = 0; w < W; ++w) {
                if (w < warp)
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
        __syncthreads();
    }
    const int HR = p.c.kv_heads * p.row_tiles;
    const long long U = (long long)s_prefix[p.c.seqs] * HR;
    const long long P = U < (long long)gridDim.x ? U : (long long)gridDim.x;
    const long long cta = blockIdx.x;
    if (cta >= P)
        return;
    const long long begin = U * cta / P, end = U * (cta + 1) / P;

    int b = 0;
    {
        int hi = p.c.seqs;  // the last b with prefix[b] * HR <= begin
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if ((long long)s_prefix[mid] * HR <= begin)
                b = mid;
            else
                hi = mid;
        }
    }

    for (long long u = begin; u < end;) {
        while ((long long)s_prefix[b + 1] * HR <= u)
            ++b;
        const Span sp = span_of<W>(p, b);
        const long long seq0 = (long long)s_prefix[b] * HR;
        const int hr = (int)((u - seq0) / sp.chunks);
        const long long unit0 = seq0 + (long long)hr * sp.chunks, unit1 = unit0 + sp.chunks;
        const int j0 = (int)(u - unit0);
        const int j1 = (int)((end < unit1 ? end : unit1) - unit0);
        const int h = hr / p.row_tiles, row0 = (hr % p.row_tiles) * ROWS;
        u = unit0 + j1;

        const int tiles_end = (sp.len + 15) >> 4;
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
        const int64_t page_stride = page_bytes * p.c.kv_heads;
        auto offset_of = [&](int i, int pg) -> int64_t {
            return (pg < 0 ? 0 : pg) * page_stride + (((tile0 + i * W) & ((1 << per_page) - 1)) << 4) * D;
        };
        uint4 kr[KC][2];       // positions g, g + 8
        uint32_t vr[4][VW];    // positions 2t, 2t + 1, 2t + 8, 2t + 9
        auto load_k = [&](int64_t at) {
#pragma unroll
            for (int c = 0; c < KC; ++c) {
                kr[c][0] = ldg_stream(k_lane + at + 64 * c);
                kr[c][1] = ldg_stream(k_lane + at + 8 * D + 64 * c);
            }
        };
        auto load_v = [&](int64_t at) {
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

        int pages = page_of(lane), pages_next = -1;
        if (n > 0) {
            const int64_t at = offset_of(0, __shfl_sync(~0u, pages, 0));
            load_k(at);
            load_v(at);
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
            const int r = row0 + nt * 8 + g;
            float top = 0.f;
            uint4 raw[KC][2];
            if (r < p.rows) {
                const int qi = r / p.group, head = h * p.group + r % p.group;
                const __nv_bfloat16 *src = p.q + ((int64_t)b * p.queries + qi) * p.q_stride + (int64_t)head * D + 16 * t;
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    raw[c][0] = __ldg(reinterpret_cast<const uint4 *>(src + 64 * c));
                    raw[c][1] = __ldg(reinterpret_cast<const uint4 *>(src + 64 * c) + 1);
                }
            } else {
#pragma unroll
                for (int c = 0; c < KC; ++c)
                    raw[c][0] = raw[c][1] = make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t w = (&raw[c][i >> 2].x)[i & 3];
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
                    const uint32_t w = (&raw[c][i >> 2].x)[i & 3];
                    qf[nt][c][i] = f16x2(bf16lo_to_f32(w) * u1 * u2, bf16hi_to_f32(w) * u1 * u2);
                }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int col = nt * 8 + 2 * t + e, rr = row0 + col;
                const int upc = __shfl_sync(~0u, up, (2 * t + e) * 4);
                factor[nt][e] = p.scale_log2 * __uint_as_float((uint32_t)(127 - upc / 2) << 23) *
                                __uint_as_float((uint32_t)(127 - (upc - upc / 2)) << 23);
                limit[nt][e] = rr < p.rows ? sp.len - p.queries + rr / p.group + 1 : 0x7fffffff;
                if (rr < p.rows)
                    lim_min = min(lim_min, limit[nt][e]);
            }
        }
        lim_min = min(lim_min, __shfl_xor_sync(~0u, lim_min, 1));
        lim_min = min(lim_min, __shfl_xor_sync(~0u, lim_min, 2));
        // tiles from here on are seen from their first position by every row
        const int lo_max = p.window > 0 ? sp.len - p.window : 0;

        float o[NT][NM][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = NEG;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int j = 0; j < NM; ++j)
                o[nt][j][0] = o[nt][j][1] = o[nt][j][2] = o[nt][j][3] = 0.f;
        }

        float lsvs = fmaxf(__log2f(svs), -64.f);
        for (int i = 0; i < n; ++i) {
            const int at32 = i & 31;
            if (at32 == 0)
                pages_next = page_of(i + 32 + lane);
            if (at32 == 16) {
                sks_next = scale_of(p.c.k_scale, pages_next);
                svs_next = scale_of(p.c.v_scale, pages_next);
            }
            const bool hole = __shfl_sync(~0u, pages, at32) < 0;
            const float sk = __shfl_sync(~0u, sks, at32), sv = __shfl_sync(~0u, svs, at32);
            const float lsv = __shfl_sync(~0u, lsvs, at32);
            const int64_t next = offset_of(i + 1, __shfl_sync(~0u, at32 == 31 ? pages_next : pages, (i + 1) & 31));

            // S^T, in two chains of MMAs where one would be long
            constexpr int CH = NT == 1 && KC > 1 ? 2 : 1;
            float s[CH][NT][4];
#pragma unroll
            for (int ch = 0; ch < CH; ++ch)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    s[ch][nt][0] = s[ch][nt][1] = s[ch][nt][2] = s[ch][nt][3] = 0.f;
#pragma unroll
            for (int w = 0; w < 4; ++w)
#pragma unroll
                for (int c = 0; c < KC; ++c) {
                    uint32_t a0, a1, a2, a3;
                    codes_to_f16<FP8>((&kr[c][0].x)[w], a0, a2);
                    codes_to_f16<FP8>((&kr[c][1].x)[w], a1, a3);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma_f16(s[c % CH][nt], a0, a1, a2, a3, qf[nt][c][2 * w], qf[nt][c][2 * w + 1]);
                }
            if (i + 1 < n)
                load_k(next);
            const int pos = (tile0 + i * W) << 4;
            const bool edge = pos + 16 > lim_min || pos < lo_max || hole;
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = s[0][nt][e];
                    if constexpr (CH == 2)
                        x += s[CH - 1][nt][e];
                    x *= factor[nt][e & 1] * sk;
                    if (edge) {
                        const int at = pos + g + 8 * (e >> 1), lim = limit[nt][e & 1];
                        if (at >= lim || (p.window > 0 && at < lim - p.window) || hole)
                            x = -INFINITY;
                    }
                    s[0][nt][e] = x;
                    grow |= x + lsv > m[nt][e & 1] + SLACK;
                }
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
            const float svp = sv * P_SCALE;
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
            // beyond the sequence's end a page may hold anything, e4m3's NaN too
            if (FP8 && edge) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (hole || pos + 2 * t + (k & 1) + 8 * (k >> 1) >= sp.len)
#pragma unroll
                        for (int w = 0; w < VW; ++w)
                            vr[k][w] = 0;
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
            if (at32 == 31) {
                pages = pages_next;
                sks = sks_next;
                svs = svs_next;
                lsvs = fmaxf(__log2f(svs), -64.f);
            }
        }

        // --- join the warps' sums
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
        __syncthreads();

        const bool whole = j0 == 0 && j1 == sp.chunks;
        const long long c0 = whole ? cta : ((unit0 + 1) * P - 1) / U, c1 = whole ? cta : (unit1 * P - 1) / U;
        // a CTA's slot 1 holds the unit that starts in it, slot 0 the one that it continues
        auto slot_of = [&](long long c) { return 2 * c + (c == c0 ? 1 : 0); };
        constexpr int PART = ROWS * (D + 2);

        auto finish = [&](int r, int at, float2 x, float mm, float ll) {  // row r, permuted index at
            const int rr = row0 + r;
            if (rr >= p.rows)
                return;
            const int qi = rr / p.group, head = h * p.group + rr % p.group;
            const int d = VB * ((at & 15) >> 1) + 2 * (at >> 4);
            const float inv = ll > 0.f ? 1.f / ll * (1.f / P_SCALE) : 0.f;
            const int64_t row = ((int64_t)b * p.queries + qi) * p.heads + head;
            *reinterpret_cast<__nv_bfloat162 *>(p.out + row * D + d) =
                __floats2bfloat162_rn(x.x * inv, x.y * inv);
            if (at == 0 && p.lse != nullptr)
                p.lse[row] = ll > 0.f ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
        };

        for (int i = tid; i < ROWS * (D / 2); i += THREADS) {
            const int r = i / (D / 2), at = 2 * (i % (D / 2));
            float mm = NEG, ll = 0.f;
            float2 x = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < W; ++w)
                mm = fmaxf(mm, s_m[w * ROWS + r]);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float a = ex2(s_m[w * ROWS + r] - mm);
                const float2 y = *reinterpret_cast<const float2 *>(s_o + (w * ROWS + r) * SM::PITCH + at);
                ll += a * s_l[w * ROWS + r];
                x.x += a * y.x;
                x.y += a * y.y;
            }
            if (whole) {
                finish(r, at, x, mm, ll);
            } else {
                float *dst = p.part + slot_of(cta) * PART;
                *reinterpret_cast<float2 *>(dst + r * D + at) = x;
                if (at == 0) {
                    dst[ROWS * D + r] = mm;
                    dst[ROWS * D + ROWS + r] = ll;
                }
            }
        }
        if (!whole) {
            // Two levels: the last CTA of each JOIN neighbours joins their sums into the first
            // one's slot, the last of those joins the unit's.
            const long long n = c1 - c0 + 1, mine = (cta - c0) / JOIN;
            const long long f0 = c0 + mine * JOIN;
            const int members = (int)(n - mine * JOIN < JOIN ? n - mine * JOIN : JOIN);
            const int joins = (int)((n + JOIN - 1) / JOIN);
            auto arrive = [&](unsigned *count, int of) -> bool {
                __syncthreads();
                if (tid == 0) {
                    __threadfence();
                    const unsigned before = atomic_add_acq_rel(count, 1u);
                    s_last = before + 1 == (unsigned)of;
                    if (s_last)
                        *count = 0;  // as the next call expects it
                    __threadfence();
                }
                __syncthreads();
                return s_last != 0;
            };
            // joins `of` slots, `step` CTAs apart from CTA f on
            auto join = [&](long long f, int step, int of, bool last) {
                for (int i = tid; i < ROWS * (D / 4); i += THREADS) {
                    const int r = i / (D / 4), at = 4 * (i % (D / 4));
                    float pm[JOIN], mm = NEG, ll = 0.f;
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int k = 0; k < JOIN; ++k) {
                        pm[k] = NEG;
                        if (k < of)
                            pm[k] = __ldcg(p.part + slot_of(f + (long long)k * step) * PART + ROWS * D + r);
                        mm = fmaxf(mm, pm[k]);
                    }
#pragma unroll
                    for (int k = 0; k < JOIN; ++k)
                        if (k < of) {
                            const float *src = p.part + slot_of(f + (long long)k * step) * PART;
                            const float a = ex2(pm[k] - mm);
                            const float4 y = __ldcg(reinterpret_cast<const float4 *>(src + r * D + at));
                            ll += a * __ldcg(src + ROWS * D + ROWS + r);
                            x.x += a * y.x;
                            x.y += a * y.y;
                            x.z += a * y.z;
                            x.w += a * y.w;
                        }
                    if (last) {
                        finish(r, at, make_float2(x.x, x.y), mm, ll);
                        finish(r, at + 2, make_float2(x.z, x.w), mm, ll);
                    } else {
                        // the first slot's other readers of m and l are this row's threads: all
                        // of a row lie in one warp's reach only if D / 4 <= 32, so they go to a
                        // copy that is written after the barrier below
                        float *dst = p.part + slot_of(f) * PART;
                        *reinterpret_cast<float4 *>(dst + r * D + at) = x;
                        if (at == 0) {
                            s_m[r] = mm;
                            s_l[r] = ll;
                        }
                    }
                }
                if (!last) {
                    __syncthreads();
                    float *dst = p.part + slot_of(f) * PART;
                    for (int r = tid; r < ROWS; r += THREADS) {
                        dst[ROWS * D + r] = s_m[r];
                        dst[ROWS * D + ROWS + r] = s_l[r];
                    }
                }
            };
            unsigned *unit_count = p.unit_count + c0;
            if (joins == 1) {
                if (arrive(unit_count, members))
                    join(f0, 1, members, true);
            } else if (arrive(p.join_count + slot_of(f0), members)) {
                join(f0, 1, members, false);
                if (arrive(unit_count, joins)) {
                    // more than JOIN * JOIN parts: fold the join's slots JOIN at a time
                    int left = joins, step = JOIN;
                    while (left > JOIN) {
                        for (int k = 0; k < left; k += JOIN) {
                            join(c0 + (long long)k * step, step, left - k < JOIN ? left - k : JOIN, false);
                            __syncthreads();
                        }
                        left = (left + JOIN - 1) / JOIN;
                        step *= JOIN;
                    }
                    join(c0, step, left, true);
                }
            }
        }
        __syncthreads();  // the sums are read
    }
}

// The variant of a call: D, the query rows of a tile and its CTAs per SM.
template <int D, int NT, bool FP8, int W, int CPS>
cudaError_t launch_variant(AttnParams &p, int sm_count, cudaStream_t stream)
{
    using SM = Smem<D, NT, W>;
    static std::atomic<unsigned long long> done{0};
    auto fn = kv8_attention_kernel<D, NT, FP8, W, CPS>;
    cudaError_t e = smem_opt_in_once(done, fn, (int)SM::bytes(MAX_SEQS));
    if (e != cudaSuccess)
        return e;
    // no more CTAs than the longest sequences that the table can hold give chunks
    const long long most = (((long long)p.c.width << p.c.page_log2) + 16 * W - 1) / (16 * W);
    const long long units = (long long)p.c.seqs * p.c.kv_heads * p.row_tiles * (most > 0 ? most : 1);
    const long long grid = units < (long long)sm_count * CPS ? units : (long long)sm_count * CPS;
    return launch_pdl(fn, dim3((unsigned)grid), dim3(32 * W), SM::bytes(p.c.seqs), stream, p);
}

constexpr int MAX_CPS = 6;  // CTAs per SM of any variant: sizes the workspace

int tile_rows(int rows, int D) { return rows <= 8 || D == 256 ? 8 : 16; }

}  // namespace

// Workspace: the counters, in the same place for every call on a device, then the partial sums.
static size_t counter_bytes(int sm_count) { return ((size_t)3 * sm_count * MAX_CPS * 4 + 255) / 256 * 256; }

size_t kv8_attention_workspace(int queries, int group, int head_dim, int sm_count)
{
    return counter_bytes(sm_count) +
           (size_t)2 * sm_count * MAX_CPS * tile_rows(queries * group, head_dim) * (head_dim + 2) * 4;
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
    const int tr = tile_rows(p.rows, c.head_dim);
    p.row_tiles = (p.rows + tr - 1) / tr;
    p.window = window;
    p.scale_log2 = scale * 1.4426950408889634f;
    p.unit_count = static_cast<unsigned *>(workspace);
    p.join_count = p.unit_count + (size_t)sm_count * MAX_CPS;
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + counter_bytes(sm_count));
#define W4Q_ATTN(D, NT, CPS)                                                          \
    return c.fp8 ? launch_variant<D, NT, true, 4, CPS>(p, sm_count, stream)           \
                 : launch_variant<D, NT, false, 4, CPS>(p, sm_count, stream)
    if (c.head_dim == 64) {
        if (tr == 8)
            W4Q_ATTN(64, 1, 6);
        W4Q_ATTN(64, 2, 4);
    }
    if (c.head_dim == 128) {
        if (tr == 8)
            W4Q_ATTN(128, 1, 4);
        W4Q_ATTN(128, 2, 3);
    }
    W4Q_ATTN(256, 1, 2);
#undef W4Q_ATTN
}

}  // namespace w4q
