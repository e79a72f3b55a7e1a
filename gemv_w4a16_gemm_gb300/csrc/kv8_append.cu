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
// rnd(code * (s / s')).  Every quotient is the correctly rounded fp32 one.
//
// What bounds it: each element is read and written once, a few dozen
// instructions an element; HBM for prompts, one launch for single tokens.
// Layout: D / 8 lanes hold a head row, 8 elements (one 16-byte load) each, so
// the norm's sum and the rotation's partners are a few shuffles away and
// nothing goes through shared memory.
#include <cuda_fp16.h>

#include "common.cuh"
#include "decode.h"
#include "kernels.h"

namespace w4q {

namespace {

struct Row {
    const __nv_bfloat16 *weight;  // null: no norm
    bool norm;                    // some row of the warp has a weight: all join the norm's shuffles
    const float *cos_sin;         // null: no rotation
    int64_t positions;
    int rot;
    bool interleaved;
    float eps;
};

__device__ __forceinline__ void unpack8(uint4 raw, float (&y)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = bf16lo_to_f32((&raw.x)[i]);
        y[2 * i + 1] = bf16hi_to_f32((&raw.x)[i]);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&y)[8])
{
    uint4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        (&r.x)[i] = *reinterpret_cast<const uint32_t *>(&h);
    }
    return r;
}

__device__ __forceinline__ void load8(const float *src, float (&y)[8])
{
    const float4 a = __ldg(reinterpret_cast<const float4 *>(src));
    const float4 b = __ldg(reinterpret_cast<const float4 *>(src) + 1);
    y[0] = a.x, y[1] = a.y, y[2] = a.z, y[3] = a.w;
    y[4] = b.x, y[5] = b.y, y[6] = b.z, y[7] = b.w;
}

// What a lane needs of the table for its 8 elements, whatever the head.
struct Angles {
    float c[8], s[8];  // interleaved: 4 of each
};

template <int D>
__device__ __forceinline__ void load_angles(const Row &p, int64_t pos, int sub, Angles &a)
{
    if (p.cos_sin == nullptr || 8 * sub >= p.rot)
        return;
    pos = pos < 0 ? 0 : (pos >= p.positions ? p.positions - 1 : pos);
    const float *t = p.cos_sin + pos * p.rot;
    const int half = p.rot / 2;
    if (p.interleaved) {
        const float4 c = __ldg(reinterpret_cast<const float4 *>(t + 4 * sub));
        const float4 s = __ldg(reinterpret_cast<const float4 *>(t + half + 4 * sub));
        a.c[0] = c.x, a.c[1] = c.y, a.c[2] = c.z, a.c[3] = c.w;
        a.s[0] = s.x, a.s[1] = s.y, a.s[2] = s.z, a.s[3] = s.w;
    } else {
        const int i = 8 * sub < half ? 8 * sub : 8 * sub - half;
        load8(t + i, a.c);
        load8(t + half + i, a.s);
    }
}

// The lane's 8 elements of a head row, normed and rotated.  All lanes of the
// warp call it together.
template <int D>
__device__ __forceinline__ void turn(const Row &p, const Angles &a, int sub, float (&y)[8])
{
    constexpr int LANES = D / 8;
    if (p.norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            ss = fmaf(y[i], y[i], ss);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1)
            ss += __shfl_xor_sync(~0u, ss, o);
        if (p.weight != nullptr) {
            const float f = rsqrtf(ss * (1.f / D) + p.eps);
            float w[8];
            unpack8(__ldg(reinterpret_cast<const uint4 *>(p.weight) + sub), w);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                y[i] = y[i] * f * w[i];
        }
    }
    if (p.cos_sin != nullptr) {
        if (p.interleaved) {
            if (8 * sub < p.rot) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float u = y[2 * i], v = y[2 * i + 1];
                    y[2 * i] = u * a.c[i] - v * a.s[i];
                    y[2 * i + 1] = v * a.c[i] + u * a.s[i];
                }
            }
        } else {
            const int half = p.rot / 16;  // lanes of half the rotated elements
            const bool first = sub < half;
            const int other = first ? sub + half : (sub < 2 * half ? sub - half : sub);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = __shfl_sync(~0u, y[i], other, LANES);
                if (sub < 2 * half)
                    y[i] = first ? y[i] * a.c[i] - v * a.s[i] : y[i] * a.c[i] + v * a.s[i];
            }
        }
    }
}

// The last b with cu[b] <= x for 0 <= x < cu[seqs] (a warp's lanes search
// together); the owner of token x.
__device__ __forceinline__ int owner_of(const int32_t *cu, int seqs, int64_t x, int lane)
{
    int lo = 0, hi = seqs;  // cu[lo] <= x < cu[hi]
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int at = lo + (lane + 1) * step;
        const bool le = at < hi && __ldg(cu + at) <= x;
        const int n = __popc(__ballot_sync(~0u, le));
        lo += n * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// --- rows of heads: [tokens][heads] strided in, contiguous out

struct HeadsIn {
    const __nv_bfloat16 *q, *k;
    __nv_bfloat16 *q_out, *k_out;
    int64_t q_stride, k_stride, tokens;
    int q_heads, k_heads;
    Row qrow, krow;
};

// One warp's task: R rows for each of its 32 / LANES groups of lanes, all of
// one token, whose angles it loads once.  `chunk` counts a token's tasks.
template <int D, int R>
__device__ __forceinline__ void heads_task(const HeadsIn &p, int64_t token, int chunk, int64_t pos, int lane)
{
    constexpr int LANES = D / 8, GROUPS = 32 / LANES;
    const int sub = lane % LANES, grp = lane / LANES;
    const int heads = p.q_heads + p.k_heads;
    uint4 raw[R];
    int head[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        head[i] = chunk * (R * GROUPS) + i * GROUPS + grp;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (head[i] < heads) {
            const bool q = head[i] < p.q_heads;
            const __nv_bfloat16 *src = q ? p.q + token * p.q_stride + (int64_t)head[i] * D
                                         : p.k + token * p.k_stride + (int64_t)(head[i] - p.q_heads) * D;
            raw[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + sub);
        }
    }
    Angles a;
    load_angles<D>(p.qrow, pos, sub, a);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const bool q = head[i] < p.q_heads;
        Row row = p.qrow;
        row.weight = q ? p.qrow.weight : p.krow.weight;
        row.norm = p.qrow.norm || p.krow.norm;
        float y[8];
        unpack8(raw[i], y);
        turn<D>(row, a, sub, y);
        if (head[i] < heads) {
            __nv_bfloat16 *dst = q ? p.q_out + (token * p.q_heads + head[i]) * D
                                   : p.k_out + (token * p.k_heads + head[i] - p.q_heads) * D;
            reinterpret_cast<uint4 *>(dst)[sub] = pack8(y);
        }
    }
}

constexpr int HEAD_WARPS = 4;

template <int D, int R>
__global__ void __launch_bounds__(32 * HEAD_WARPS) qk_norm_rope_kernel(const HeadsIn p, const int32_t *pos,
                                                                       int chunks)
{
    pdl_wait();
    pdl_launch_dependents();
    const int64_t task = (int64_t)blockIdx.x * HEAD_WARPS + (threadIdx.x >> 5);
    const int64_t token = task / chunks;
    if (token >= p.tokens)
        return;
    heads_task<D, R>(p, token, (int)(task % chunks), pos ? pos[token] : token, threadIdx.x & 31);
}

// --- codes

// max |y| / top and the codes of 8 elements, for either format
template <bool FP8>
__device__ __forceinline__ uint2 encode8(const float (&y)[8], float s)
{
    uint32_t w[2] = {0, 0};
    if (s > 0.f) {
        if constexpr (FP8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint16_t h;
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                    : "=h"(h)
                    : "f"(__fdiv_rn(y[2 * i + 1], s)), "f"(__fdiv_rn(y[2 * i], s)));
                w[i >> 1] |= (uint32_t)h << (16 * (i & 1));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = fminf(fmaxf(rintf(__fdiv_rn(y[i], s)), -127.f), 127.f);
                w[i >> 2] |= ((uint32_t)(int)q & 0xFFu) << (8 * (i & 3));
            }
        }
    }
    return make_uint2(w[0], w[1]);
}

template <bool FP8>
__device__ __forceinline__ void decode8(uint2 c, float (&y)[8])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = ((i & 2) ? c.y : c.x) >> (16 * (i & 1));
        if constexpr (FP8) {
            uint32_t f;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(f) : "h"((uint16_t)h));
            const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&f));
            y[2 * i] = v.x;
            y[2 * i + 1] = v.y;
        } else {
            y[2 * i] = (float)(int8_t)(h & 0xFF);
            y[2 * i + 1] = (float)(int8_t)((h >> 8) & 0xFF);
        }
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
        y[i] *= r;
    return encode8<FP8>(y, 1.f);
}

template <int LANES>
__device__ __forceinline__ float max_abs(const float (&y)[8])
{
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        a = fmaxf(a, fabsf(y[i]));
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1)
        a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
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

// One new token per sequence: a warp writes one (sequence, kv head) row of K or
// V, its groups of D / 8 lanes computing the same row; the first blocks take
// the query heads.  A page whose scale grows (one token in n + 1 with n before
// it, on gaussian rows) is read and written back 4 KB at a time, so that its
// loads wait for memory together.
template <int D, bool FP8>
__global__ void __launch_bounds__(32 * HEAD_WARPS) kv8_append_one_kernel(const AppendParams p)
{
    constexpr int LANES = D / 8, BATCH = 8;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int sub = lane % LANES;
    if ((int)blockIdx.x < p.head_blocks) {
        const int64_t task = (int64_t)blockIdx.x * HEAD_WARPS + warp;
        const int64_t token = task / p.head_chunks;
        if (token < p.tokens)
            heads_task<D, 1>(p.heads, token, (int)(task % p.head_chunks), (int64_t)p.c.lens[token] - 1, lane);
        return;
    }
    int unit = (int)(blockIdx.x - p.head_blocks) * HEAD_WARPS + warp;
    const int per = p.c.kv_heads * p.c.seqs;
    const bool value = unit >= per;
    unit -= value ? per : 0;
    if (unit >= per)
        return;
    const int b = unit / p.c.kv_heads, h = unit % p.c.kv_heads;
    const int64_t pos = (int64_t)p.c.lens[b] - 1;
    if (pos < 0 || (pos >> p.c.page_log2) >= p.c.width)
        return;
    const uint4 raw = __ldcs(reinterpret_cast<const uint4 *>((value ? p.v + b * p.v_stride : p.k + b * p.k_stride) +
                                                             (int64_t)h * D) + sub);
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
    if (!value) {
        Angles a;
        load_angles<D>(p.krow, pos, sub, a);
        turn<D>(p.krow, a, sub, y);
    }
    old = __shfl_sync(~0u, old, 0);
    const float s = fmaxf(__fdiv_rn(max_abs<LANES>(y), FP8 ? 448.f : 127.f), old);
    uint8_t *codes = (value ? p.c.v : p.c.k) + ((ph << p.c.page_log2) * D);
    if (lane < LANES)
        reinterpret_cast<uint2 *>(codes + (int64_t)slot * D)[lane] = encode8<FP8>(y, s);
    if (lane == 0)
        *scale = s;
    if (slot > 0 && s > old) {
        const float r = __fdiv_rn(old, s);
        uint4 *held = reinterpret_cast<uint4 *>(codes);
        const int n = slot * (D / 16);
        for (int i0 = lane; i0 < n; i0 += 32 * BATCH) {
            uint4 c[BATCH];
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (i0 + 32 * i < n)
                    c[i] = held[i0 + 32 * i];
#pragma unroll
            for (int i = 0; i < BATCH; ++i)
                if (i0 + 32 * i < n) {
                    const uint2 lo = recode8<FP8>(make_uint2(c[i].x, c[i].y), r);
                    const uint2 hi = recode8<FP8>(make_uint2(c[i].z, c[i].w), r);
                    held[i0 + 32 * i] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                }
        }
    }
}

// Any number of new tokens per sequence: one CTA writes the part of one page
// (of one kv head, K or V) that they fill.  Page j of the new tokens of
// sequence b is number cu[b] / page + 2 b + j: at least as many numbers lie
// between one sequence's first and the next one's as it can touch pages, so
// tokens / page + 2 seqs CTAs per head cover every case and the ones without
// a page leave.
constexpr int PAGE_THREADS = 256;

template <int D, int PL, bool FP8>
__global__ void __launch_bounds__(PAGE_THREADS) kv8_append_kernel(const AppendParams p)
{
    constexpr int LANES = D / 8, AT_ONCE = PAGE_THREADS / LANES, PAGE = 1 << PL;
    constexpr int R = PAGE > AT_ONCE ? PAGE / AT_ONCE : 1;
    __shared__ float s_max[PAGE_THREADS / 32];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, sub = lane % LANES;
    if ((int)blockIdx.x < p.head_blocks) {
        const int64_t task = (int64_t)blockIdx.x * (PAGE_THREADS / 32) + warp;
        const int64_t token = task / p.head_chunks;
        if (token < p.tokens) {
            const int b = owner_of(p.cu, p.c.seqs, token, lane);
            const int64_t pos = (int64_t)p.c.lens[b] - p.cu[b + 1] + token;
            heads_task<D, 2>(p.heads, token, (int)(task % p.head_chunks), pos, lane);
        }
        return;
    }
    int64_t unit = blockIdx.x - p.head_blocks;
    const bool value = unit % 2;
    unit /= 2;
    const int h = (int)(unit % p.c.kv_heads);
    unit /= p.c.kv_heads;
    int b = -1;
    for (int i0 = 0; i0 < p.c.seqs; i0 += PAGE_THREADS) {
        const int i = i0 + tid;
        b += __syncthreads_count(i < p.c.seqs && (int64_t)(__ldg(p.cu + i) >> PL) + 2 * i <= unit);
    }
    if (b < 0)
        return;
    const int64_t first = __ldg(p.cu + b), count = __ldg(p.cu + b + 1) - first;
    const int64_t len = p.c.lens[b], before = len - count;
    const int64_t start = before > 0 ? before : 0;
    const int64_t pg = (start >> PL) + (unit - ((first >> PL) + 2 * b));
    if (count <= 0 || (pg << PL) >= len || pg >= p.c.width)
        return;
    const int page = __ldg(p.c.table + (int64_t)b * p.c.width + pg);
    if ((unsigned)page >= (unsigned)p.c.blocks)
        return;
    const int64_t pos0 = pg << PL;
    const int held = (int)(before > pos0 ? before - pos0 : 0);  // earlier tokens of the page
    const int64_t ph = (int64_t)page * p.c.kv_heads + h;
    float *scale = (value ? p.c.v_scale : p.c.k_scale) + ph;
    const float old = held > 0 ? *scale : 0.f;

    Row row = p.krow;
    if (value) {
        row.norm = false;
        row.cos_sin = nullptr;
    }
    auto is_new = [&](int slot, int64_t &token) {
        const int64_t pos = pos0 + slot;
        token = first + pos - before;
        return slot < PAGE && pos >= start && pos < len && token >= 0 && token < p.tokens;
    };
    uint4 raw[R] = {};
    float top = 0.f;
    auto values = [&](int i, float (&y)[8]) {
        Angles a;
        load_angles<D>(row, pos0 + i * AT_ONCE + tid / LANES, sub, a);
        unpack8(raw[i], y);
        turn<D>(row, a, sub, y);
    };
#pragma unroll
    for (int i = 0; i < R; ++i) {
        int64_t token;
        raw[i] = make_uint4(0, 0, 0, 0);
        if (is_new(i * AT_ONCE + tid / LANES, token))
            raw[i] = __ldcs(reinterpret_cast<const uint4 *>((value ? p.v + token * p.v_stride : p.k + token * p.k_stride) +
                                                            (int64_t)h * D) + sub);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float y[8];
        values(i, y);
        top = fmaxf(top, max_abs<32>(y));
    }
    if (lane == 0)
        s_max[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < PAGE_THREADS / 32; ++w)
        top = fmaxf(top, s_max[w]);
    const float s = fmaxf(__fdiv_rn(top, FP8 ? 448.f : 127.f), old);
    uint2 *codes = reinterpret_cast<uint2 *>((value ? p.c.v : p.c.k) + ((ph << PL) * D)) + sub;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int slot = i * AT_ONCE + tid / LANES;
        int64_t token;
        float y[8];
        values(i, y);
        if (is_new(slot, token))
            codes[slot * LANES] = encode8<FP8>(y, s);
        else if (slot < held && s > old)
            codes[slot * LANES] = recode8<FP8>(codes[slot * LANES], __fdiv_rn(old, s));
    }
    if (tid == 0)
        *scale = s;
}

// The values that the cache stands for: the last cu[b + 1] - cu[b] positions
// of each sequence, one after the other.
template <int D, bool FP8>
__global__ void __launch_bounds__(32 * HEAD_WARPS) kv8_read_kernel(const Kv8 c, const int32_t *cu, int64_t tokens,
                                                                   __nv_bfloat16 *k_out, __nv_bfloat16 *v_out,
                                                                   int chunks)
{
    constexpr int LANES = D / 8, GROUPS = 32 / LANES;
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31, sub = lane % LANES;
    const int64_t task = (int64_t)blockIdx.x * HEAD_WARPS + (threadIdx.x >> 5);
    const int64_t token = task / chunks;
    if (token >= tokens)
        return;
    const int b = cu ? owner_of(cu, c.seqs, token, lane) : (int)token;
    const int64_t pos = (int64_t)c.lens[b] - (cu ? cu[b + 1] - token : 1);
    const int h = (int)(task % chunks) * GROUPS + lane / LANES;
    if (h >= c.kv_heads)
        return;
    int64_t page = -1;
    if (pos >= 0 && pos < c.lens[b] && (pos >> c.page_log2) < c.width)
        page = __ldg(c.table + (int64_t)b * c.width + (pos >> c.page_log2));
    float k[8] = {}, v[8] = {};
    if (page >= 0 && page < c.blocks) {
        const int64_t ph = page * c.kv_heads + h;
        const int64_t at = ((ph << c.page_log2) + (pos & ((1 << c.page_log2) - 1))) * LANES + sub;
        decode8<FP8>(__ldg(reinterpret_cast<const uint2 *>(c.k) + at), k);
        decode8<FP8>(__ldg(reinterpret_cast<const uint2 *>(c.v) + at), v);
        const float sk = c.k_scale[ph], sv = c.v_scale[ph];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            k[i] *= sk;
            v[i] *= sv;
        }
    }
    const int64_t to = (token * c.kv_heads + h) * LANES + sub;
    reinterpret_cast<uint4 *>(k_out)[to] = pack8(k);
    reinterpret_cast<uint4 *>(v_out)[to] = pack8(v);
}

Row row_of(const HeadPrep &prep, const void *weight)
{
    return Row{static_cast<const __nv_bfloat16 *>(weight), weight != nullptr, prep.cos_sin, prep.positions, prep.rot,
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
    const int chunks = chunks_of(heads, D, few ? 1 : 4);
    const int64_t blocks = (in.tokens * chunks + HEAD_WARPS - 1) / HEAD_WARPS;
    if (few)
        return launch_pdl(qk_norm_rope_kernel<D, 1>, dim3((unsigned)blocks), dim3(32 * HEAD_WARPS), 0, stream, in,
                          pos, chunks);
    return launch_pdl(qk_norm_rope_kernel<D, 4>, dim3((unsigned)blocks), dim3(32 * HEAD_WARPS), 0, stream, in, pos,
                      chunks);
}

template <int D, bool FP8>
cudaError_t append(AppendParams &p, cudaStream_t stream)
{
    const bool one = p.cu == nullptr;
    const int warps = one ? HEAD_WARPS : PAGE_THREADS / 32;
    if (p.heads.q_heads > 0) {
        p.head_chunks = chunks_of(p.heads.q_heads, D, one ? 1 : 2);
        p.head_blocks = (int)((p.tokens * p.head_chunks + warps - 1) / warps);
    }
    if (one) {
        const int64_t units = 2LL * p.c.seqs * p.c.kv_heads;
        return launch_pdl(kv8_append_one_kernel<D, FP8>,
                          dim3((unsigned)(p.head_blocks + (units + HEAD_WARPS - 1) / HEAD_WARPS)),
                          dim3(32 * HEAD_WARPS), 0, stream, p);
    }
    const int64_t units = ((p.tokens >> p.c.page_log2) + 2LL * p.c.seqs) * p.c.kv_heads * 2;
    const dim3 grid((unsigned)(p.head_blocks + units)), block(PAGE_THREADS);
    switch (p.c.page_log2) {
    case 4: return launch_pdl(kv8_append_kernel<D, 4, FP8>, grid, block, 0, stream, p);
    case 5: return launch_pdl(kv8_append_kernel<D, 5, FP8>, grid, block, 0, stream, p);
    case 6: return launch_pdl(kv8_append_kernel<D, 6, FP8>, grid, block, 0, stream, p);
    default: return launch_pdl(kv8_append_kernel<D, 7, FP8>, grid, block, 0, stream, p);
    }
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
