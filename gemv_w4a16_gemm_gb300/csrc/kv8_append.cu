// kv8_append.cu -- norms of query and key heads with their position rotation
// in one pass, and the writer and the reader of the paged 8-bit cache.
//
// Head row x of D elements, weight w, position p with the table's cosines c and
// sines s of rot / 2 angles:
//     y = x / sqrt(mean x^2 + eps) * w           (with a weight)
//     (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s)
// for the pairs (i, i + rot / 2), or (2i, 2i + 1) interleaved, i < rot / 2; the
// elements from rot on stay.  All of it in fp32, rounded once.
//
// Cache page of one head, holding codes and one fp32 scale: the new tokens' rows
// that fall into it give
//     s' = max(s, max |y| / top)   (s = 0 for a page without earlier tokens;
//                                   top = 127 for int8, 448 for e4m3)
// and the codes rnd(y / s'); where s' > s the earlier codes become
// rnd(code * (s / s')).  Every quotient is the correctly rounded fp32 one.  A NaN
// or infinite element: e4m3 keeps it as its code NaN and leaves it out of the
// maximum; int8 has no such code, so s' is NaN and the page's head reads as NaN.
//
// What bounds it: each element is read and written once, some fifty
// instructions for a lane's 8 of them.  Rotation of prompts: HBM.  The writer of
// prompts: no unit is full (64% of the issue slots, ALU 54%, HBM 40%), its warps
// wait for loads and for each other's results.  Single tokens: one launch and
// its chain of dependent loads.  Layout: D / 8 lanes hold a head row.  A lane has two groups of 4
// elements, one from each half of the rotated part (or 8 beyond it), so both
// partners of its pairs and their 4 angles are its own: the norm's sum is the
// only thing that lanes exchange.  Measured: 8191 tokens of 56 heads of 128
// rotated in 42.9 us, 81% of the measured copy bandwidth; 5862 tokens of 5
// sequences (8 kv heads, 32 query heads, e4m3) written in 37.8 us for the 19.9 of
// their bytes and read back in 9.2 for 5.3, 16 bytes a lane in flight; 64 x 1
// written in 3.8 us, written and read (1881 tokens) in 8.4.  (Query heads in a launch of their own after the
// pages': 55 us for 5 x 2000; a warp going through several heads of a page: 50.)
#include <cuda_fp16.h>

#include <cfloat>

#include "common.cuh"
#include "decode.h"
#include "kernels.h"

namespace w4q {

namespace {

struct Row {
    const __nv_bfloat16 *weight;  // null: no norm
    const float *cos_sin;         // null: no rotation
    int64_t positions;
    int rot;
    bool interleaved;
    float eps;
};

// A lane's elements of a row: a[0..3] from offset first on, a[4..7] from second on.
struct Where {
    int first, second;
};

template <int D>
__device__ __forceinline__ Where elements_of(const Row &p, int sub)
{
    if (p.interleaved)
        return {8 * sub, 8 * sub + 4};
    const int turned = p.rot / 8;  // lanes of the rotated part
    if (sub < turned)
        return {4 * sub, p.rot / 2 + 4 * sub};
    return {8 * sub, 8 * sub + 4};
}

struct Raw {
    uint2 a, b;
};

__device__ __forceinline__ Raw load_raw(const __nv_bfloat16 *row, Where w)
{
    return {__ldg(reinterpret_cast<const uint2 *>(row + w.first)), __ldg(reinterpret_cast<const uint2 *>(row + w.second))};
}

__device__ __forceinline__ void unpack8(Raw r, float (&y)[8])
{
    y[0] = bf16lo_to_f32(r.a.x), y[1] = bf16hi_to_f32(r.a.x), y[2] = bf16lo_to_f32(r.a.y), y[3] = bf16hi_to_f32(r.a.y);
    y[4] = bf16lo_to_f32(r.b.x), y[5] = bf16hi_to_f32(r.b.x), y[6] = bf16lo_to_f32(r.b.y), y[7] = bf16hi_to_f32(r.b.y);
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ void store_row(__nv_bfloat16 *row, Where w, const float (&y)[8])
{
    *reinterpret_cast<uint2 *>(row + w.first) = make_uint2(bf16_pair(y[0], y[1]), bf16_pair(y[2], y[3]));
    *reinterpret_cast<uint2 *>(row + w.second) = make_uint2(bf16_pair(y[4], y[5]), bf16_pair(y[6], y[7]));
}

// What a lane needs for every row of a kind and a position: the norm's weights
// and the angles of its pairs.
struct Weights {
    float w[8];
};
__device__ __forceinline__ Weights load_weights(const Row &p, Where at)
{
    Weights v = {};
    if (p.weight != nullptr)
        unpack8(load_raw(p.weight, at), v.w);
    return v;
}

struct Angles {
    float4 c, s;
};
__device__ __forceinline__ Angles load_angles(const Row &p, int64_t pos, int sub)
{
    Angles a = {};
    if (p.cos_sin != nullptr && 8 * sub < p.rot) {
        pos = pos < 0 ? 0 : (pos >= p.positions ? p.positions - 1 : pos);
        const float *t = p.cos_sin + pos * p.rot + 4 * sub;
        a.c = __ldg(reinterpret_cast<const float4 *>(t));
        a.s = __ldg(reinterpret_cast<const float4 *>(t + p.rot / 2));
    }
    return a;
}

// Two fp32 operations in one instruction, rounded as one by one: (a, b) = (a x, b y) and (a, b) = (x u + a, y v + b).
__device__ __forceinline__ void mul2(float &a, float &b, float x, float y)
{
    asm("{\n\t.reg .b64 p, q;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\tmul.rn.f32x2 p, p, q;\n\t"
        "mov.b64 {%0, %1}, p;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(x), "f"(y));
}
__device__ __forceinline__ void fma2(float &a, float &b, float x, float y, float u, float v)
{
    asm("{\n\t.reg .b64 p, q, r;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\tmov.b64 r, {%0, %1};\n\t"
        "fma.rn.f32x2 r, p, q, r;\n\tmov.b64 {%0, %1}, r;\n\t}"
        : "+f"(a), "+f"(b)
        : "f"(x), "f"(y), "f"(u), "f"(v));
}

// The lane's 8 elements of a head row, normed and rotated.  All lanes of the
// warp call it together.
template <int D>
__device__ __forceinline__ void turn(const Row &p, const Weights &w, const Angles &a, int sub, float (&y)[8])
{
    constexpr int LANES = D / 8;
    if (p.weight != nullptr) {
        float ss = 0.f, st = 0.f;
#pragma unroll
        for (int i = 0; i < 8; i += 2)
            fma2(ss, st, y[i], y[i + 1], y[i], y[i + 1]);
        ss += st;
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1)
            ss += __shfl_xor_sync(~0u, ss, o);
        const float f = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            mul2(y[i], y[i + 1], f, f);
            mul2(y[i], y[i + 1], w.w[i], w.w[i + 1]);
        }
    }
    if (p.cos_sin != nullptr && 8 * sub < p.rot) {
        const float c[4] = {a.c.x, a.c.y, a.c.z, a.c.w}, s[4] = {a.s.x, a.s.y, a.s.z, a.s.w};
        if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = y[2 * i], v = y[2 * i + 1];
                y[2 * i] = u * c[i] - v * s[i];
                y[2 * i + 1] = v * c[i] + u * s[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float u0 = y[i], u1 = y[i + 1], v0 = y[4 + i], v1 = y[5 + i];
                mul2(y[i], y[i + 1], c[i], c[i + 1]);
                fma2(y[i], y[i + 1], v0, v1, -s[i], -s[i + 1]);
                mul2(y[4 + i], y[5 + i], c[i], c[i + 1]);
                fma2(y[4 + i], y[5 + i], u0, u1, s[i], s[i + 1]);
            }
        }
    }
}

// The last b in [0, seqs) with key(b) <= x, for a rising key with key(0) <= x;
// a warp's lanes search together.
template <class Key>
__device__ __forceinline__ int last_at_most(Key key, int seqs, int64_t x, int lane)
{
    int lo = 0, hi = seqs;  // key(lo) <= x < key(hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const bool le = at < hi && key(at) <= x;
        lo += __popc(__ballot_sync(~0u, le)) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// The sequence that token x of those laid out by the prefix sums cu belongs to.
__device__ __forceinline__ int owner_of(const int32_t *cu, int seqs, int64_t x, int lane)
{
    return last_at_most([cu](int b) { return (int64_t)__ldg(cu + b); }, seqs, x, lane);
}

// --- rows of heads: [tokens][heads] strided in, contiguous out

struct HeadsIn {
    const __nv_bfloat16 *q, *k;
    __nv_bfloat16 *q_out, *k_out;
    int64_t q_stride, k_stride, tokens;
    int q_heads, k_heads;
    Row qrow, krow;
};

// One warp's task: R rows for each of its 32 / LANES groups of lanes, heads of
// one kind and one token, whose weights and angles it loads once.  A token has
// q_chunks tasks of query heads, then those of the key heads.
template <int D, int R>
struct HeadsTask {
    static constexpr int LANES = D / 8, GROUPS = 32 / LANES, ROWS = R * GROUPS;
    Raw raw[R];
    const __nv_bfloat16 *weight;
    __nv_bfloat16 *out;
    int head0, heads;

    // the rows' loads; what follows may wait for the position meanwhile
    __device__ __forceinline__ void load(const HeadsIn &p, int64_t token, int chunk, int q_chunks, int lane)
    {
        const bool q = chunk < q_chunks;
        heads = q ? p.q_heads : p.k_heads;
        head0 = (q ? chunk : chunk - q_chunks) * ROWS + lane / LANES;
        const Where at = elements_of<D>(p.qrow, lane % LANES);
        const __nv_bfloat16 *row = q ? p.q + token * p.q_stride : p.k + token * p.k_stride;
        out = q ? p.q_out + token * heads * D : p.k_out + token * heads * D;
        weight = q ? p.qrow.weight : p.krow.weight;
#pragma unroll
        for (int i = 0; i < R; ++i)  // heads past the last are its copies, and are not stored
            raw[i] = load_raw(row + (int64_t)min(head0 + i * GROUPS, heads - 1) * D, at);
    }
    __device__ __forceinline__ void store(const HeadsIn &p, int64_t pos, int lane)
    {
        const int sub = lane % LANES;
        Row row = p.qrow;
        row.weight = weight;
        const Where at = elements_of<D>(row, sub);
        const Angles a = load_angles(row, pos, sub);
        const Weights w = load_weights(row, at);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            float y[8];
            unpack8(raw[i], y);
            turn<D>(row, w, a, sub, y);
            if (head0 + i * GROUPS < heads)
                store_row(out + (int64_t)(head0 + i * GROUPS) * D, at, y);
        }
    }
};

constexpr int HEAD_WARPS = 4;

template <int D, int R>
__global__ void __launch_bounds__(32 * HEAD_WARPS) qk_norm_rope_kernel(const HeadsIn p, const int32_t *pos,
                                                                       int q_chunks, int chunks)
{
    const int64_t task = (int64_t)blockIdx.x * HEAD_WARPS + (threadIdx.x >> 5);
    const unsigned token = (unsigned)task / (unsigned)chunks;
    pdl_wait();
    pdl_launch_dependents();
    if (token >= p.tokens)
        return;
    HeadsTask<D, R> t;
    t.load(p, token, (int)(task - (int64_t)token * chunks), q_chunks, threadIdx.x & 31);
    t.store(p, pos ? (int64_t)__ldg(pos + token) : (int64_t)token, threadIdx.x & 31);
}

// --- codes

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi)
{
    uint16_t h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(hi), "f"(lo));
    return h;
}

// The codes of y / 1, |y| <= 127 (int8).
template <bool FP8>
__device__ __forceinline__ uint2 encode8(const float (&y)[8])
{
    uint32_t w[2] = {0, 0};
    if constexpr (FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i >> 1] |= e4m3_pair(y[2 * i], y[2 * i + 1]) << (16 * (i & 1));
    } else {
        // 1.5 2^23 + y rounds y to an integer (half to even) whose low byte is the code; |y| <= 127
        uint32_t q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[i] = __float_as_uint(__fadd_rn(y[i], 12582912.f));
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = prmt(prmt(q[4 * i], q[4 * i + 1], 0x0040u), prmt(q[4 * i + 2], q[4 * i + 3], 0x0040u), 0x5410u);
    }
    return make_uint2(w[0], w[1]);
}

// The codes of the correctly rounded quotients y / s, for |y| / top <= s or y NaN (e4m3).  A
// quotient costs a dozen instructions; y times the rounded reciprocal lies
// within 2^-22 of it and gives the same code except next to a rounding's edge,
// where the quotient decides (int8: act_code8; e4m3: both ends of the interval
// 2^-21 wide are converted and have to agree).
template <bool FP8>
__device__ __forceinline__ uint2 encode8(const float (&y)[8], float s)
{
    float q[8];
    if (!(s > 0.f)) {
        if constexpr (!FP8)
            return make_uint2(0u, 0u);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            q[i] = fabsf(y[i]) * 0.f;  // 0, and NaN's code
        return encode8<FP8>(q);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = y[i];
    if constexpr (FP8) {
        const float r = __frcp_rn(s), lo = r * (1.f - 0x1p-21f), hi = r * (1.f + 0x1p-21f);
        uint32_t a[2] = {0, 0}, b[2] = {0, 0};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            a[i >> 1] |= e4m3_pair(q[2 * i] * lo, q[2 * i + 1] * lo) << (16 * (i & 1));
            b[i >> 1] |= e4m3_pair(q[2 * i] * hi, q[2 * i + 1] * hi) << (16 * (i & 1));
        }
        if (a[0] != b[0] || a[1] != b[1] || !(s >= 0x1p-125f)) {  // below that the reciprocal overflows
#pragma unroll
            for (int i = 0; i < 8; ++i)
                q[i] = __fdiv_rn(q[i], s);
            return encode8<true>(q);
        }
        return make_uint2(a[0], a[1]);
    } else {
        act_code8(q, s);
        return encode8<false>(q);
    }
}

template <bool FP8>
__device__ __forceinline__ void decode8(uint2 c, float (&y)[8])
{
    if constexpr (FP8) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t f;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"((uint16_t)(((i & 2) ? c.y : c.x) >> (16 * (i & 1)))));
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&f));
            y[2 * i] = v.x;
            y[2 * i + 1] = v.y;
        }
    } else {
        // the byte with its sign flipped under 0x4B0000 is 2^23 + 128 + code
#pragma unroll
        for (int i = 0; i < 8; ++i)
            y[i] = __uint_as_float(prmt((i < 4 ? c.x : c.y) ^ 0x80808080u, 0x4B000000u, 0x7440u + (i & 3))) - 8388736.f;
    }
}

// Earlier tokens' codes under the page's new scale, r = s / s'.
template <bool FP8>
__device__ __forceinline__ uint2 recode8(uint2 c, float r)
{
    float y[8];
    decode8<FP8>(c, y);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = __fmul_rn(y[i], r);  // rounded by itself: not fused with the rounding to a code
    return encode8<FP8>(y);
}

// Infinities become NaN.
__device__ __forceinline__ void mark(float (&y)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i)
        y[i] = fabsf(y[i]) <= FLT_MAX ? y[i] : NAN;
}

// max(a, b), NaN if either is
__device__ __forceinline__ float max_nan(float a, float b)
{
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// The largest |y| of a lane's elements and of a group of lanes: NaN if one is (with IGNORE, of the others).
template <bool IGNORE>
__device__ __forceinline__ float max_abs(const float (&y)[8])
{
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        a = IGNORE ? fmaxf(a, fabsf(y[i])) : max_nan(a, fabsf(y[i]));
    return a;
}
template <int LANES>
__device__ __forceinline__ float max_of(float a)
{
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
        a = max_nan(a, __shfl_xor_sync(~0u, a, o));
    return a;
}

struct AppendParams {
    Kv8 c;
    const __nv_bfloat16 *k, *v;
    int64_t k_stride, v_stride, tokens;
    const int32_t *cu;
    HeadsIn heads;  // the queries (k_heads = 0), q_heads = 0: none
    Row krow;
    int head_chunks;
    int head_blocks;
};

// A lane's codes of a row of D, where its elements are.
__device__ __forceinline__ void store_codes(uint8_t *row, Where w, uint2 c)
{
    *reinterpret_cast<uint32_t *>(row + w.first) = c.x;
    *reinterpret_cast<uint32_t *>(row + w.second) = c.y;
}

// Rewrites n 16-byte groups of codes under the page's new scale, by `all`
// threads of which this is `me`, eight groups a thread at a time, so that their
// loads wait for memory together.
template <bool FP8>
__device__ __forceinline__ void recode(uint4 *held, int n, int me, int all, float r)
{
    constexpr int BATCH = 8;
    for (int i0 = me; i0 < n; i0 += all * BATCH) {
        uint4 c[BATCH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (i0 + all * i < n)
                c[i] = held[i0 + all * i];
#pragma unroll
        for (int i = 0; i < BATCH; ++i)
            if (i0 + all * i < n) {
                const uint2 lo = recode8<FP8>(make_uint2(c[i].x, c[i].y), r);
                const uint2 hi = recode8<FP8>(make_uint2(c[i].z, c[i].w), r);
                held[i0 + all * i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
    }
}

// One new token per sequence: a warp writes one (sequence, kv head) row of K or
// V, its groups of D / 8 lanes computing the same row; the first blocks take
// the query heads.  A page whose scale grows (one token in n + 1 with n before
// it, on gaussian rows) is read and written back.
template <int D, bool FP8>
__global__ void __launch_bounds__(32 * HEAD_WARPS) kv8_append_one_kernel(const AppendParams p)
{
    constexpr int LANES = D / 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane % LANES;
    pdl_wait();
    pdl_launch_dependents();
    if ((int)blockIdx.x < p.head_blocks) {
        const unsigned task = blockIdx.x * HEAD_WARPS + warp, token = task / (unsigned)p.head_chunks;
        if (token < p.tokens) {
            HeadsTask<D, 1> t;
            t.load(p.heads, token, (int)(task - token * p.head_chunks), p.head_chunks, lane);
            t.store(p.heads, (int64_t)p.c.lens[token] - 1, lane);
        }
        return;
    }
    int unit = (int)(blockIdx.x - p.head_blocks) * HEAD_WARPS + warp;
    const int per = p.c.kv_heads * p.c.seqs;
    const bool value = unit >= per;
    unit -= value ? per : 0;
    if (unit >= per)
        return;
    const int b = (int)((unsigned)unit / (unsigned)p.c.kv_heads), h = unit - b * p.c.kv_heads;
    const int64_t pos = (int64_t)p.c.lens[b] - 1;
    const Where at = elements_of<D>(p.krow, sub);
    const Raw raw = load_raw((value ? p.v + b * p.v_stride : p.k + b * p.k_stride) + (int64_t)h * D, at);
    if (pos < 0 || (pos >> p.c.page_log2) >= p.c.width)
        return;
    const int page = __ldg(p.c.table + (int64_t)b * p.c.width + (pos >> p.c.page_log2));
    if ((unsigned)page >= (unsigned)p.c.blocks)
        return;
    const int64_t ph = (int64_t)page * p.c.kv_heads + h;
    const int slot = (int)(pos & ((1 << p.c.page_log2) - 1));
    float *scale = (value ? p.c.v_scale : p.c.k_scale) + ph;
    float old = 0.f;
    if (lane == 0 && slot > 0)
        old = *scale;
    float y[8];
    unpack8(raw, y);
    if (!value)
        turn<D>(p.krow, load_weights(p.krow, at), load_angles(p.krow, pos, sub), sub, y);
    old = __shfl_sync(~0u, old, 0);
    float top = max_of<LANES>(max_abs<false>(y));
    if (!(top <= FLT_MAX)) {  // (of the whole warp: its groups of lanes hold the same row)
        mark(y);
        top = FP8 ? max_of<LANES>(max_abs<true>(y)) : NAN;
    }
    const float s = max_nan(__fdiv_rn(top, FP8 ? 448.f : 127.f), old);
    uint8_t *codes = (value ? p.c.v : p.c.k) + ((ph << p.c.page_log2) * D);
    if (lane < LANES)
        store_codes(codes + (int64_t)slot * D, at, encode8<FP8>(y, s));
    if (lane == 0)
        *scale = s;
    if (slot > 0 && s > old)
        recode<FP8>(reinterpret_cast<uint4 *>(codes), slot * (D / 16), lane, 32, __fdiv_rn(old, s));
}

// Any number of new tokens per sequence: `share` warps (a power of two) write
// the part of one page (of one kv head, K or V) that they fill.  Page j of the
// new tokens of sequence b is number cu[b] / page + 2 b + j: at least as many
// numbers lie between one sequence's first and the next one's as it can touch
// pages, so tokens / page + 2 seqs numbers cover every case and the ones
// without a page are left.  The scale needs every row and the codes need the
// scale: up to 2 rows of a group of lanes stay in registers in between, more
// are computed again.  (64 registers a thread, so that the query heads' blocks
// of the same launch keep 32 warps an SM busy with loads.)
constexpr int PAGE_WARPS = 8;

template <int D, bool FP8>
__global__ void __launch_bounds__(32 * PAGE_WARPS, 4) kv8_append_kernel(const AppendParams p, int share)
{
    constexpr int LANES = D / 8, GROUPS = 32 / LANES, R = 2;
    __shared__ float s_max[PAGE_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane % LANES;
    pdl_wait();
    pdl_launch_dependents();
    // the pages' blocks come first: they take longest
    const int page_blocks = gridDim.x - p.head_blocks;
    if ((int)blockIdx.x >= page_blocks) {
        const int64_t task = (int64_t)(blockIdx.x - page_blocks) * PAGE_WARPS + warp;
        const unsigned token = (unsigned)task / (unsigned)p.head_chunks;
        if (token < p.tokens) {
            HeadsTask<D, 4> t;
            t.load(p.heads, token, (int)(task - (int64_t)token * p.head_chunks), p.head_chunks, lane);
            const int b = owner_of(p.cu, p.c.seqs, token, lane);
            t.store(p.heads, (int64_t)p.c.lens[b] - __ldg(p.cu + b + 1) + token, lane);
        }
        return;
    }
    // the unit of this warp and its place among the unit's warps; K and V of a page, then its heads
    const unsigned unit = (blockIdx.x * PAGE_WARPS + warp) / (unsigned)share;
    const int part = warp & (share - 1), page_log2 = p.c.page_log2, page = 1 << page_log2;
    const bool value = unit & 1;
    const int number = (int)((unit >> 1) / (unsigned)p.c.kv_heads), h = (int)((unit >> 1) - number * (unsigned)p.c.kv_heads);
    const int32_t *cu = p.cu;
    bool live = number < (p.tokens >> page_log2) + 2 * p.c.seqs;
    const int b = last_at_most([cu, page_log2](int i) { return (int64_t)(__ldg(cu + i) >> page_log2) + 2 * i; }, p.c.seqs,
                               number, lane);
    const int64_t first = __ldg(cu + b), count = __ldg(cu + b + 1) - first;
    const int64_t len = p.c.lens[b], before = len - count;
    const int64_t start = before > 0 ? before : 0;
    const int64_t pg = (start >> page_log2) + (number - ((first >> page_log2) + 2 * b)), pos0 = pg << page_log2;
    live = live && count > 0 && pg >= (start >> page_log2) && pos0 < len && pg < p.c.width;
    const int block = live ? __ldg(p.c.table + (int64_t)b * p.c.width + pg) : -1;
    live = (unsigned)block < (unsigned)p.c.blocks;
    // the new slots lo .. hi - 1 of the page; the ones below lo hold earlier tokens
    const int lo = (int)(start > pos0 ? start - pos0 : 0);
    const int hi = live ? (int)(len - pos0 < page ? len - pos0 : page) : 0;
    const int64_t ph = (live ? (int64_t)block : 0) * p.c.kv_heads + h;
    float *scale = (value ? p.c.v_scale : p.c.k_scale) + ph;

    Row row = p.krow;
    if (value) {
        row.weight = nullptr;
        row.cos_sin = nullptr;
    }
    const Where at = elements_of<D>(p.krow, sub);
    const __nv_bfloat16 *src = (value ? p.v : p.k) + (int64_t)h * D;
    const int64_t stride = value ? p.v_stride : p.k_stride, token0 = first + pos0 - before;
    // Row i of batch n of this group of lanes is a slot of its own; the first new slots go to all warps.
    auto slot_of = [&](int n, int i) { return lo + part + share * ((n * R + i) * GROUPS + lane / LANES); };
    auto any = [&](int n, int i) { return lo + part + share * (n * R + i) * GROUPS < hi; };  // of the warp's
    auto is_token = [&](int slot) { return slot < hi && token0 + slot >= 0 && token0 + slot < p.tokens; };
    const Weights weights = load_weights(row, at);
    float y[R][8];
    auto batch = [&](int n) {
        Raw raw[R] = {};
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (is_token(slot_of(n, i)))
                raw[i] = load_raw(src + (token0 + slot_of(n, i)) * stride, at);
#pragma unroll
        for (int i = 0; i < R; ++i) {
            unpack8(raw[i], y[i]);
            if (any(n, i))
                turn<D>(row, weights, load_angles(row, pos0 + slot_of(n, i), sub), sub, y[i]);
        }
    };
    float old = 0.f;
    if (lane == 0 && lo > 0 && hi > 0)
        old = *scale;
    const bool kept = !any(1, 0);
    float top = 0.f;
    for (int n = 0; n == 0 || any(n, 0); ++n) {
        batch(n);
#pragma unroll
        for (int i = 0; i < R; ++i)
            top = max_nan(top, max_abs<false>(y[i]));
    }
    top = max_of<32>(top);
    const bool odd = !(top <= FLT_MAX);  // a row of this warp holds NaN or infinity
    auto mark_all = [&]() {
#pragma unroll
        for (int i = 0; i < R; ++i)
            mark(y[i]);
    };
    if (odd) {
        top = FP8 ? 0.f : NAN;
        for (int n = 0; FP8 && (n == 0 || any(n, 0)); ++n) {
            if (!kept)
                batch(n);
            mark_all();
#pragma unroll
            for (int i = 0; i < R; ++i)
                top = fmaxf(top, max_abs<true>(y[i]));
        }
        top = max_of<32>(top);
    }
    old = __shfl_sync(~0u, old, 0);
    if (share > 1) {
        if (lane == 0)
            s_max[warp] = top;
        __syncthreads();
        for (int w = 0; w < share; ++w)
            top = max_nan(top, s_max[warp - part + w]);
    }
    if (hi == 0)
        return;
    const float s = max_nan(__fdiv_rn(top, FP8 ? 448.f : 127.f), old);
    uint8_t *codes = (value ? p.c.v : p.c.k) + ((ph << page_log2) * D);
    for (int n = 0; n == 0 || any(n, 0); ++n) {
        if (!kept) {
            batch(n);
            if (FP8 && odd)
                mark_all();
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
            if (is_token(slot_of(n, i)))
                store_codes(codes + (int64_t)slot_of(n, i) * D, at, encode8<FP8>(y[i], s));
    }
    if (part == 0 && lane == 0)
        *scale = s;
    if (lo > 0 && s > old)
        recode<FP8>(reinterpret_cast<uint4 *>(codes), lo * (D / 16), part * 32 + lane, 32 * share, __fdiv_rn(old, s));
}

// The values that the cache stands for: the last cu[b + 1] - cu[b] positions
// of each sequence, one after the other; 8 codes a lane.
template <int D, bool FP8>
__global__ void __launch_bounds__(32 * HEAD_WARPS) kv8_read_kernel(const Kv8 c, const int32_t *cu, int64_t tokens,
                                                                   __nv_bfloat16 *k_out, __nv_bfloat16 *v_out,
                                                                   int chunks)
{
    constexpr int LANES = D / 8, GROUPS = 32 / LANES;
    const int lane = threadIdx.x & 31, sub = lane % LANES;
    const int64_t task = (int64_t)blockIdx.x * HEAD_WARPS + (threadIdx.x >> 5);
    const unsigned token = (unsigned)task / (unsigned)chunks;
    pdl_wait();
    pdl_launch_dependents();
    if (token >= tokens)
        return;
    const int b = cu ? owner_of(cu, c.seqs, token, lane) : (int)token;
    const int64_t len = c.lens[b], pos = len - (cu ? __ldg(cu + b + 1) - (int64_t)token : 1);
    const int h = (int)(task - (int64_t)token * chunks) * GROUPS + lane / LANES;
    if (h >= c.kv_heads)
        return;
    int page = -1;
    if (pos >= 0 && pos < len && (pos >> c.page_log2) < c.width)
        page = __ldg(c.table + (int64_t)b * c.width + (pos >> c.page_log2));
    float k[8] = {}, v[8] = {};
    if ((unsigned)page < (unsigned)c.blocks) {
        const int64_t ph = (int64_t)page * c.kv_heads + h;
        const int64_t at = ((ph << c.page_log2) + (pos & ((1 << c.page_log2) - 1))) * LANES + sub;
        const uint2 kc = __ldg(reinterpret_cast<const uint2 *>(c.k) + at), vc = __ldg(reinterpret_cast<const uint2 *>(c.v) + at);
        const float sk = c.k_scale[ph], sv = c.v_scale[ph];
        decode8<FP8>(kc, k);
        decode8<FP8>(vc, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            k[i] *= sk;
            v[i] *= sv;
        }
    }
    const Where w = {8 * sub, 8 * sub + 4};
    const int64_t to = ((int64_t)token * c.kv_heads + h) * D;
    store_row(k_out + to, w, k);
    store_row(v_out + to, w, v);
}

Row row_of(const HeadPrep &prep, const void *weight)
{
    return Row{static_cast<const __nv_bfloat16 *>(weight), prep.cos_sin, prep.positions, prep.rot,
               prep.interleaved, prep.eps};
}

int chunks_of(int heads, int D, int R)
{
    const int n = R * (32 / (D / 8));
    return (heads + n - 1) / n;
}

template <int D>
cudaError_t norm_rope(const HeadsIn &in, const int32_t *pos, cudaStream_t stream)
{
    // Four rows per group of lanes keep 64 bytes a lane in flight and load a token's angles once
    // for all of them; with few tokens one row each spreads the call over more SMs.
    const int heads = in.q_heads + in.k_heads;
    const bool few = in.tokens * heads * (D / 8) < 152LL * 2048;
    const int R = few ? 1 : 4, q_chunks = chunks_of(in.q_heads, D, R), chunks = q_chunks + chunks_of(in.k_heads, D, R);
    const dim3 grid((unsigned)((in.tokens * chunks + HEAD_WARPS - 1) / HEAD_WARPS)), block(32 * HEAD_WARPS);
    return launch_pdl(few ? qk_norm_rope_kernel<D, 1> : qk_norm_rope_kernel<D, 4>, grid, block, 0, stream, in, pos,
                      q_chunks, chunks);
}

template <int D, bool FP8>
cudaError_t append(AppendParams &p, cudaStream_t stream)
{
    if (p.cu == nullptr) {
        if (p.heads.q_heads > 0) {
            p.head_chunks = chunks_of(p.heads.q_heads, D, 1);
            p.head_blocks = (int)((p.tokens * p.head_chunks + HEAD_WARPS - 1) / HEAD_WARPS);
        }
        const int64_t units = 2LL * p.c.seqs * p.c.kv_heads;
        return launch_pdl(kv8_append_one_kernel<D, FP8>,
                          dim3((unsigned)(p.head_blocks + (units + HEAD_WARPS - 1) / HEAD_WARPS)),
                          dim3(32 * HEAD_WARPS), 0, stream, p);
    }
    if (p.heads.q_heads > 0) {
        p.head_chunks = chunks_of(p.heads.q_heads, D, 4);
        p.head_blocks = (int)((p.tokens * p.head_chunks + PAGE_WARPS - 1) / PAGE_WARPS);
    }
    // Warps per page: as many as hold a full page in registers, one where a sequence brings few
    // tokens (64 sequences with one token: 14 us with 8, 6.4 us with one).
    int share = 1;
    if (p.tokens >= 8LL * p.c.seqs)
        while (share < PAGE_WARPS && (D << p.c.page_log2) > 512 * share)
            share *= 2;
    const int64_t units = ((p.tokens >> p.c.page_log2) + 2LL * p.c.seqs) * p.c.kv_heads * 2, per = PAGE_WARPS / share;
    return launch_pdl(kv8_append_kernel<D, FP8>, dim3((unsigned)(p.head_blocks + (units + per - 1) / per)),
                      dim3(32 * PAGE_WARPS), 0, stream, p, share);
}

template <int D>
cudaError_t read(const Kv8 &c, const int32_t *cu, int64_t tokens, void *k_out, void *v_out, cudaStream_t stream)
{
    const int chunks = chunks_of(c.kv_heads, D, 1);
    const dim3 grid((unsigned)((tokens * chunks + HEAD_WARPS - 1) / HEAD_WARPS)), block(32 * HEAD_WARPS);
    return launch_pdl(c.fp8 ? kv8_read_kernel<D, true> : kv8_read_kernel<D, false>, grid, block, 0, stream, c, cu,
                      tokens, static_cast<__nv_bfloat16 *>(k_out), static_cast<__nv_bfloat16 *>(v_out), chunks);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const void *q, const void *k, int64_t tokens, int q_heads, int k_heads,
                                int head_dim, int64_t q_stride, int64_t k_stride, const HeadPrep &prep,
                                const int32_t *pos, void *q_out, void *k_out, cudaStream_t stream)
{
    HeadsIn in = {static_cast<const __nv_bfloat16 *>(q), static_cast<const __nv_bfloat16 *>(k),
                  static_cast<__nv_bfloat16 *>(q_out), static_cast<__nv_bfloat16 *>(k_out),
                  q_stride, k_stride, tokens, q_heads, k_heads,
                  row_of(prep, prep.q_weight), row_of(prep, prep.k_weight)};
    return head_dim == 64 ? norm_rope<64>(in, pos, stream)
           : head_dim == 128 ? norm_rope<128>(in, pos, stream) : norm_rope<256>(in, pos, stream);
}

cudaError_t launch_kv8_append(const Kv8 &c, const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                              int64_t tokens, const int32_t *cu, const void *q, int64_t q_stride, int q_heads,
                              void *q_out, const HeadPrep &prep, cudaStream_t stream)
{
    AppendParams p = {};
    p.c = c;
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.tokens = tokens;
    p.cu = cu;
    p.krow = row_of(prep, prep.k_weight);
    p.heads.q = static_cast<const __nv_bfloat16 *>(q);
    p.heads.q_out = static_cast<__nv_bfloat16 *>(q_out);
    p.heads.q_stride = q_stride;
    p.heads.tokens = tokens;
    p.heads.q_heads = q_heads;
    p.heads.qrow = row_of(prep, prep.q_weight);
    p.heads.krow = p.heads.qrow;
    if (c.head_dim == 64)
        return c.fp8 ? append<64, true>(p, stream) : append<64, false>(p, stream);
    if (c.head_dim == 128)
        return c.fp8 ? append<128, true>(p, stream) : append<128, false>(p, stream);
    return c.fp8 ? append<256, true>(p, stream) : append<256, false>(p, stream);
}

cudaError_t launch_kv8_read(const Kv8 &c, const int32_t *cu, int64_t tokens, void *k_out, void *v_out,
                            cudaStream_t stream)
{
    return c.head_dim == 64 ? read<64>(c, cu, tokens, k_out, v_out, stream)
           : c.head_dim == 128 ? read<128>(c, cu, tokens, k_out, v_out, stream)
                               : read<256>(c, cu, tokens, k_out, v_out, stream);
}

}  // namespace w4q
