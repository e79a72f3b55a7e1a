// verify.cu -- drafted tokens checked against the target's logits, and the token
// that follows them.
//
// Row i of a sequence holds the logits l after its first i drafts, p = softmax(l / T):
//     draft d_i is accepted while u_i q_i(d_i) < p_i(d_i)     (q = 1 without drafts' probabilities)
//     at the first one that is not: the v with the largest (p_i(v) - q_i(v))+ / e(v)
//     behind the last draft:        the v with the largest p(v) / e(v)
// with given uniform u and exponential e: v / e for positive weights v is largest at
// an index with probability v / sum v, so no cumulative sum is needed, and the CTAs
// of a row join by a maximum.  T = 0: p is 1 at the largest logit.
//
// Two launches.  The first forms each row's maximum, its place and the sum of
// exp((l - max) / T), a row's vocabulary cut among CTAs.  In the second, every CTA of
// a sequence joins those, decides which drafts are accepted, and goes over its cut of
// the one row that matters; the last of them writes the result.  Without drafts the race
// needs no sum: the largest l / T - log e is found in the first launch, and the second only
// joins (256 x 128256: 37 us, 56 with a second pass).  There the best so far is kept as l and
// log e, not as a score relative to some maximum, and two of them are compared by their
// difference, as if exactly: equal ones stay equal, and how a row is cut decides nothing.
//
// What bounds it: the logits of all rows and, for one row a sequence, q and e, from
// HBM; for few sequences the chain of dependent loads of two launches.  Loads are 16
// bytes wide and aligned.  Rows that do not begin on 16 bytes (an odd vocabulary) have
// their ragged ends read one by one; where logits, e and q lie differently, the others'
// loads take a neighbour more and are shifted to one's (256 x 50257 without drafts 38.8 us
// with single elements, 18.4 so, as much as 50264; 64 x 5 rows of 151937 42.5 and 36.5).
#include <cfloat>
#include <climits>

#include "common.cuh"
#include "decode.h"

namespace w4q {

namespace {

constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int MAX_PARTS = 32;    // cuts of a row: one a lane where they are joined
constexpr int PART_MIN = 8192;   // elements that a CTA's beginning and end are worth: 64 x 5 rows of 151936 cut in
                                 // 2 (one wave) take 35 us, in 1, 4, 7, 14: 46, 37, 38, 43
constexpr int MAX_QUERIES = 64;
// CTAs of an SM in the launches.  (Racing, bf16: 256 x 128256 37 us, 65 with 3, which spills; fp32:
// 64 x 32000 7.2 us, 256 x 128256 49; 7.8 and 46 with 4, 7.1 and 55 with 2.  Else bf16: 64 x 5 rows
// of 151936 34.9, 35.7 with 4; fp32, which spills with 5: 64 x 4 rows of 32000 14.3, 16.1 and 14.9
// with 3 and 5.)
constexpr int PICK_CTAS = 3;
constexpr int rows_ctas(bool f32) { return f32 ? 4 : 5; }
constexpr int race_ctas(bool f32) { return f32 ? 3 : 2; }
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct VerifyArgs {
    const void *logits;
    int64_t stride;
    const int32_t *drafts, *counts;
    const float *probs, *temperature, *uniforms, *noise;
    int32_t *tokens, *accepted;
    float *logprobs;
    int seqs, queries, vocab, parts1, parts2;
    bool raced;          // no drafts: the first launch does it all but the joins
    float4 *stats;       // [rows][parts1]: maximum, sum, place of the maximum (of greedy rows)
    float2 *best;        // [seqs][parts2]: score and place; [seqs][parts1] where the first launch raced: logit
                         // and log2 e of the best, whose place stands in stats
    unsigned *arrived;   // [seqs]
};

// NaN counts as -infinity, +infinity as the type's largest number.
template <bool F32>
__device__ __forceinline__ float clean(float x)
{
    return fminf(fmaxf(x, -INFINITY), F32 ? FLT_MAX : 0x1.FEp127f);
}

template <bool F32>
__device__ __forceinline__ float logit(const void *base, int64_t i)
{
    if (F32)
        return clean<true>(__ldg(static_cast<const float *>(base) + i));
    const uint16_t b = __ldg(static_cast<const uint16_t *>(base) + i);
    return clean<false>(__uint_as_float((uint32_t)b << 16));
}

// The elements of a 16-byte load, cleaned: 8 bf16 or 4 fp32.
template <bool F32>
__device__ __forceinline__ void spread(uint4 r, float (&x)[F32 ? 4 : 8])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (F32) {
            x[j] = clean<true>(__uint_as_float(w[j]));
        } else {
            uint32_t v;
            asm("max.bf16x2 %0, %1, %2;\n\tmin.bf16x2 %0, %0, %3;" : "=&r"(v) : "r"(w[j]), "r"(0xFF80FF80u), "r"(0x7F7F7F7Fu));
            x[2 * j] = bf16lo_to_f32(v);
            x[2 * j + 1] = bf16hi_to_f32(v);
        }
    }
}

__device__ __forceinline__ float exp2_of(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A sequence's temperature: log2(e) / T, so that exp((l - m) / T) = 2^((l - m) c);
// greedy for T <= 0 (and NaN), whose probabilities are then those of T = 1.
struct Heat {
    float c;
    bool greedy;
};
__device__ __forceinline__ Heat heat_of(const VerifyArgs &p, int seq)
{
    const float t = p.temperature != nullptr ? __ldg(p.temperature + seq) : 1.f;
    if (!(t > 0.f))
        return {LOG2E, true};
    return {fminf(fmaxf(__fdiv_rn(LOG2E, t), 0x1p-100f), 0x1p100f), false};
}

__device__ __forceinline__ int count_of(const VerifyArgs &p, int seq)
{
    const int d = p.queries - 1;
    return p.counts != nullptr ? min(max(__ldg(p.counts + seq), 0), d) : d;
}

// Maximum and sum of 2^((x - max) c).
struct Sum {
    float m, z;
};
__device__ __forceinline__ Sum joined(const Sum &a, const Sum &b, float c)
{
    Sum r;
    r.m = fmaxf(a.m, b.m);
    const float base = r.m == -INFINITY ? 0.f : r.m;
    r.z = a.z * exp2_of((a.m - base) * c) + b.z * exp2_of((b.m - base) * c);
    return r;
}
__device__ __forceinline__ Sum joined_lanes(Sum s, float c)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
        s = joined(s, {__shfl_xor_sync(0xffffffffu, s.m, o), __shfl_xor_sync(0xffffffffu, s.z, o)}, c);
    return s;
}

// A row's, with the maximum's first place (of greedy rows).
struct Stat {
    float m, z;
    int at;
};

// The numbers of a 16-byte load as they are.
template <bool F32>
__device__ __forceinline__ void raw(uint4 r, float (&x)[F32 ? 4 : 8])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if constexpr (F32) {
            x[j] = __uint_as_float(w[j]);
        } else {
            x[2 * j] = bf16lo_to_f32(w[j]);
            x[2 * j + 1] = bf16hi_to_f32(w[j]);
        }
    }
}

// The largest number of U loads; NaN is passed over.
template <bool F32, int U>
__device__ __forceinline__ float top_of(const uint4 (&r)[U])
{
    if constexpr (F32) {
        float t = -INFINITY;
#pragma unroll
        for (int i = 0; i < U; ++i)
            t = fmaxf(t, fmaxf(fmaxf(__uint_as_float(r[i].x), __uint_as_float(r[i].y)), fmaxf(__uint_as_float(r[i].z), __uint_as_float(r[i].w))));
        return t;
    } else {
        uint32_t t = 0xFF80FF80u;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const uint32_t w[4] = {r[i].x, r[i].y, r[i].z, r[i].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                asm("max.bf16x2 %0, %0, %1;" : "+r"(t) : "r"(w[j]));
        }
        return fmaxf(bf16lo_to_f32(t), bf16hi_to_f32(t));
    }
}

// N elements from the d-th (0 to 3) of N / 4 + 1 loads.
template <int N>
__device__ __forceinline__ void shifted(const float4 (&r)[N / 4 + 1], int d, float (&x)[N])
{
    float t[N + 4];
#pragma unroll
    for (int i = 0; i < N / 4 + 1; ++i)
        t[4 * i] = r[i].x, t[4 * i + 1] = r[i].y, t[4 * i + 2] = r[i].z, t[4 * i + 3] = r[i].w;
#pragma unroll
    for (int i = 0; i < N + 2; ++i)
        t[i] = d & 1 ? t[i + 1] : t[i];
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = d & 2 ? t[i + 2] : t[i];
}
// 8 bf16 from the d-th (0 to 7) of two loads.
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int d)
{
    uint32_t t[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 7; ++i)
        t[i] = d & 2 ? t[i + 1] : t[i];
#pragma unroll
    for (int i = 0; i < 5; ++i)
        t[i] = d & 4 ? t[i + 2] : t[i];
    const int bits = 16 * (d & 1);
    return make_uint4(__funnelshift_r(t[0], t[1], bits), __funnelshift_r(t[1], t[2], bits), __funnelshift_r(t[2], t[3], bits),
                      __funnelshift_r(t[3], t[4], bits));
}

// The best of a thread's elements, score = log2 of p / e up to the row's sum, relative to the
// thread's maximum.
struct Pick {
    float score;
    int at;
};

// The larger score, the lower place among equal ones.
__device__ __forceinline__ Pick better(const Pick &a, const Pick &b)
{
    return a.score > b.score || (a.score == b.score && (unsigned)a.at < (unsigned)b.at) ? a : b;
}
__device__ __forceinline__ Pick best_lane(Pick a)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        a = better(a, {__shfl_xor_sync(0xffffffffu, a.score, o), __shfl_xor_sync(0xffffffffu, a.at, o)});
    return a;
}

// The best of some elements in a race without a sum: the largest x c - log2 e.
struct Runner {
    float x, log_e;  // -infinity and 0 where there is none
    int at;
};
// By how much a leads b; exact in its sign but for the last of 45 bits of the terms.
__device__ __forceinline__ float lead(const Runner &a, const Runner &b, float c)
{
    const float dx = a.x - b.x, dl = a.log_e - b.log_e, p = __fmul_rn(dx, c), r = p - dl;
    if (fabsf(r) >= 0x1p-20f * (fabsf(p) + fabsf(dl)))
        return r;
    // r is exact: what the differences and the product were rounded by
    const float tx = dx - a.x, tl = dl - a.log_e;
    const float ex = (a.x - (dx - tx)) - (b.x + tx), el = (a.log_e - (dl - tl)) - (b.log_e + tl);
    return r + ((fmaf(dx, c, -p) + ex * c) - el);
}
// The one that leads, the lower place where none does.
__device__ __forceinline__ Runner better(const Runner &a, const Runner &b, float c)
{
    const float d = lead(a, b, c);
    return d > 0.f || (!(d < 0.f) && (unsigned)a.at < (unsigned)b.at) ? a : b;
}
// Below `score` by more than two fp32 scores (x - ref) c - log2 e of equal elements differ, each
// of whose terms is at most 150 above it and is rounded three times.
__device__ __forceinline__ float below(float score) { return score - (fabsf(score) * 0x1p-21f + 0x1p-14f); }
// The best of the lanes, by scores relative to any number `ref`, of which hardly ever two are so near.
// (All of it by `better` took 0.4 us.)
__device__ __forceinline__ Runner best_lane(Runner a, float ref, float c)
{
    const float score = (a.x - ref) * c - a.log_e;
    float top = score;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const unsigned near = __ballot_sync(0xffffffffu, score > below(top));
    if (__popc(near) == 1) {
        const int from = __ffs(near) - 1;
        return {__shfl_sync(0xffffffffu, a.x, from), __shfl_sync(0xffffffffu, a.log_e, from), __shfl_sync(0xffffffffu, a.at, from)};
    }
    if (top > -INFINITY)
#pragma unroll 1
        for (int o = 16; o > 0; o >>= 1)
            a = better(a, {__shfl_xor_sync(0xffffffffu, a.x, o), __shfl_xor_sync(0xffffffffu, a.log_e, o), __shfl_xor_sync(0xffffffffu, a.at, o)}, c);
    return a;
}

// 1 / e enters as -log2 e, so that the race of a whole row needs no sum.
__device__ __forceinline__ float log2_of(float x)
{
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A row that is raced over, its noise, and where this CTA's loads of it end.
struct RaceRow {
    const void *row;
    const float *e;
    int end;
};

// Element j of consecutive loads.
template <int N>
__device__ __forceinline__ float element(const float4 (&e)[N], int j)
{
    const float4 f = e[j / 4];
    return j % 4 == 0 ? f.x : (j % 4 == 1 ? f.y : (j % 4 == 2 ? f.z : f.w));
}

// Adds U loads of a row, the first of which begins at element `at`, the others `step`
// elements further on each, to a thread's sums; RACE: and to its warp's race, with the same
// elements' e.
// batch: `at` of the loads with the first of its maxima.  With every element cleaned by itself
// the pass over 64 x 5 rows of 151936 executed 15 instructions an element and was bound by them
// (25.5 us); 7.8 so, in 17.  A NaN or +infinity is found by what it makes of the
// sum, and the loads are cleaned only then.  more: many follow, and the lanes of a warp share their
// best (in every batch, 17 x 50257 took 6.4 us, 5.6 so).
template <bool F32, int U, bool RACE>
__device__ __forceinline__ void add_loads(Sum &s, const uint4 (&r)[U], int at, int step, bool more, const Heat &heat, int &batch, Runner &best,
                                          const float4 (&e)[RACE ? U : 1][F32 ? 1 : 2], const RaceRow &race)
{
    constexpr int W = F32 ? 4 : 8;
    float top = top_of<F32, U>(r);
    const bool odd = top == INFINITY;
    top = fminf(top, F32 ? FLT_MAX : 0x1.FEp127f);
    const float m = fmaxf(s.m, top), ref = m == -INFINITY ? 0.f : m;
    float2 sum[2] = {};
    const float2 minus = {-ref, -ref}, c = {heat.c, heat.c};
    // scores relative to the thread's maximum so far, of which those above `bar` may lead the warp's best
    float score[RACE ? U * W : 1], high = -INFINITY;
    const float bar = RACE ? below((best.x - ref) * heat.c - best.log_e) : 0.f;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        float x[W];
        raw<F32>(r[i], x);
#pragma unroll
        for (int j = 0; j < W; j += 2) {
            const float2 t = mul2(add2({x[j], x[j + 1]}, minus), c);
            sum[j / 2 & 1] = add2(sum[j / 2 & 1], {exp2_of(t.x), exp2_of(t.y)});
            if constexpr (RACE) {
                const float4 f = e[i][j / 4];
                score[i * W + j] = t.x - log2_of(j % 4 == 0 ? f.x : f.z);
                score[i * W + j + 1] = t.y - log2_of(j % 4 == 0 ? f.y : f.w);
                high = fmaxf(high, fmaxf(score[i * W + j], score[i * W + j + 1]));
            }
        }
    }
    const float2 both = add2(sum[0], sum[1]);
    float z = both.x + both.y;
    bool found = false;
    if (odd || z != z) {
        z = 0.f;
        found = true;
#pragma unroll 1
        for (int i = 0; i < U; ++i) {
            uint4 one = r[0];
#pragma unroll
            for (int k = 1; k < U; ++k)
                if (i == k)
                    one = r[k];
            float x[W];
            spread<F32>(one, x);
#pragma unroll
            for (int j = 0; j < W; ++j) {
                z += exp2_of((x[j] - ref) * heat.c);
            }
        }
    }
    if constexpr (RACE) {
        // Seldom in a long row, whose warps' lanes share their best: with a thread's own some lane
        // came in at most batches.
        if (__any_sync(0xffffffffu, found || high > bar)) {
            const float least = fmaxf(bar, below(high));
            Runner top = {-INFINITY, 0.f, -1};
            unsigned near = 0u;
#pragma unroll
            for (int i = U - 1; i >= 0; --i) {
                float x[W];
                raw<F32>(r[i], x);
#pragma unroll
                for (int j = W - 1; j >= 0; --j)
                    if (score[i * W + j] > least) {
                        near |= 1u << (i * W + j);
                        top = {x[j], element(e[i], j), at + i * step + j};
                    }
            }
            top.log_e = log2_of(top.log_e);
            near = found ? (1u << (U * W)) - 1u : (high > bar ? near : 0u);
            if (__popc(near) == 1 && below(below(high)) > bar) {
                best = top;
            } else {  // one by one, loaded again: a short code for what is rare
#pragma unroll 1
                for (; near != 0u; near &= near - 1u) {
                    const int k = __ffs(near) - 1, v = at + k / W * step + k % W;
                    if (v < race.end) {
                        const Runner one = {logit<F32>(race.row, v), log2_of(__ldg(race.e + v)), v};
                        if ((one.x - ref) * heat.c - one.log_e > bar)
                            best = better(one, best, heat.c);
                    }
                }
            }
            if (more) {
                const float first = __shfl_sync(0xffffffffu, best.x, 0);
                best = best_lane(best, first > -INFINITY ? first : 0.f, heat.c);
            }
        }
    }
    if (m > s.m) {
        batch = at;
        s.z *= exp2_of((s.m - m) * heat.c);
        s.m = m;
    }
    s.z += z;
}

// How the first launch races: not at all; rows of e lie in 16-byte loads as those of the
// logits do; they lie anyhow.
enum { NO_RACE, RACE_ALIGNED, RACE_SHIFTED };

// e of a load's elements, the first of what was loaded or the d-th.
template <int N>
__device__ __forceinline__ void place_e(float4 (&e)[N], const float4 (&r)[N], int)
{
#pragma unroll
    for (int j = 0; j < N; ++j)
        e[j] = r[j];
}
template <int N>
__device__ __forceinline__ void place_e(float4 (&e)[N], const float4 (&r)[N + 1], int d)
{
    float x[4 * N];
    shifted<4 * N>(r, d, x);
#pragma unroll
    for (int j = 0; j < N; ++j)
        e[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
}

template <int N>
struct Int {  // N as a type
    static constexpr int value = N;
};

template <bool F32, int RACE>  // RACE: there are no drafts
__global__ void __launch_bounds__(THREADS, RACE ? race_ctas(F32) : rows_ctas(F32)) verify_rows_kernel(const VerifyArgs p)
{
    constexpr int W = F32 ? 4 : 8, U = RACE ? 2 : 4;         // elements of a load, loads at a time
    constexpr int E = W / 4, L = E + (RACE == RACE_SHIFTED);  // a load's e, and what is loaded for them
    __shared__ Sum part[WARPS];
    __shared__ Runner part_best[WARPS];
    __shared__ int place;
    const int row = blockIdx.x / p.parts1, cut = blockIdx.x % p.parts1;
    const int seq = row / p.queries, query = row % p.queries;
    // Loads are aligned: the row is elements a .. end - 1 of those from `base` on.  This CTA
    // has loads lo .. hi - 1 of it, whole ones; the row's ragged ends are read one by one.
    const int64_t begin = row * p.stride, noise = (int64_t)seq * p.vocab;
    const int a = (int)(begin % W), end = a + p.vocab;
    const int64_t base = begin - a;
    // shifted, the loads of e reach up to 3 elements before the logits' and 4 behind them
    const int apart = RACE == RACE_SHIFTED;
    const int first = (a + W - 1) / W + apart, whole = max(end / W - apart - first, 0);
    const int lo = first + (int)((int64_t)cut * whole / p.parts1), hi = first + (int)((int64_t)(cut + 1) * whole / p.parts1);
    const uint4 *l = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(p.logits) + base * (16 / W));
    const int d = RACE == RACE_SHIFTED ? (int)((noise - a) & 3) : 0;
    const float *e = p.noise + (noise - a - d);
    pdl_wait();
    // only now: the second launch reads its other inputs before it waits for this one
    pdl_launch_dependents();
    uint4 r[U];
    float4 re[RACE ? U : 1][L];
    const uint32_t none = F32 ? 0xFF800000u : 0xFF80FF80u;
    auto load = [&](int from) {  // loads `from` on, U of each thread's
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int v = from + i * THREADS + threadIdx.x;
            r[i] = v < hi ? __ldg(l + v) : make_uint4(none, none, none, none);
            if constexpr (RACE != NO_RACE)
#pragma unroll
                for (int j = 0; j < L; ++j)
                    re[i][j] = v < hi ? __ldg(reinterpret_cast<const float4 *>(e + W * v) + j) : make_float4(1.f, 1.f, 1.f, 1.f);
        }
    };
    load(lo);  // the first loads go out before what says how they count
    if (query == 0 && cut == 0 && threadIdx.x == 0)
        p.arrived[seq] = 0u;
    const Heat heat = heat_of(p, seq);
    if (query > count_of(p, seq))
        return;
    Sum s = {-INFINITY, 0.f};
    int batch = 0;
    Runner best = {-INFINITY, 0.f, -1};
    const RaceRow race = {static_cast<const uint8_t *>(p.logits) + begin * (16 / W), p.noise + noise, hi * W - a};
    constexpr int G = 4;  // loads at a time of a greedy row that is not raced over
    if (RACE != NO_RACE && heat.greedy) {
        // Its noise does not count, and only the first loads' was asked for (256 x 128256 37.0 us with
        // all of it, 18.2 so; 64 of fp32 15.0 and 9.8).
        uint4 g[G];
        auto fetch = [&](int from) {
#pragma unroll
            for (int i = 0; i < G; ++i) {
                const int v = from + i * THREADS + threadIdx.x;
                g[i] = v < hi ? __ldg(l + v) : make_uint4(none, none, none, none);
            }
        };
        auto at = [&](int from) { return (from + (int)threadIdx.x) * W - a; };
        const float4 unused[1][F32 ? 1 : 2] = {};
        int from = lo + U * THREADS;
        fetch(from);
        add_loads<F32, U, false>(s, r, at(lo), THREADS * W, false, heat, batch, best, unused, race);
        for (; from < hi; from += G * THREADS) {
            uint4 now[G];
#pragma unroll
            for (int i = 0; i < G; ++i)
                now[i] = g[i];
            fetch(from + G * THREADS);
            add_loads<F32, G, false>(s, now, at(from), THREADS * W, false, heat, batch, best, unused, race);
        }
    } else {
        for (int from = lo; from < hi; from += U * THREADS) {
            uint4 now[U];
            float4 ne[RACE ? U : 1][E];
#pragma unroll
            for (int i = 0; i < U; ++i) {
                now[i] = r[i];
                if constexpr (RACE != NO_RACE)
                    place_e<E>(ne[i], re[i], d);
            }
            if (from + U * THREADS < hi)
                load(from + U * THREADS);
            const int at = (from + (int)threadIdx.x) * W - a;
            // the first n of them: with only all or one, 80 rows of 32000 took 8.7 us instead of 8.2
            auto add = [&](auto n) {
                constexpr int N = decltype(n)::value;
                uint4 some[N];
                float4 se[RACE ? N : 1][E];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    some[i] = now[i];
                    if constexpr (RACE != NO_RACE)
                        place_e<E>(se[i], ne[i], 0);
                }
                add_loads<F32, N, RACE != NO_RACE>(s, some, at, THREADS * W, hi - from > 5 * U * THREADS, heat, batch, best, se, race);
            };
            if (U > 2 && hi - from > 2 * THREADS)
                add(Int<U>());
            else if (hi - from > THREADS)
                add(Int<2>());
            else
                add(Int<1>());
        }
    }
    // the elements before the first whole load and behind the last one: fewer than 4 W
    const int head = min(first * W, end) - a, tail = first * W < end ? end - (first + whole) * W : 0;
    const bool odd = cut == 0 && (int)threadIdx.x < head + tail;  // this thread has one
    const int odd_at = (int)threadIdx.x < head ? threadIdx.x : p.vocab - tail + threadIdx.x - head;
    if (odd) {
        const float x = logit<F32>(p.logits, begin + odd_at);
        s = joined(s, {x, x == -INFINITY ? 0.f : 1.f}, heat.c);
        if (RACE && !heat.greedy) {
            const Runner one = {x, log2_of(__ldg(p.noise + noise + odd_at)), odd_at};
            if (x > -INFINITY && one.log_e < INFINITY)
                best = better(one, best, heat.c);
        }
    }
    const float m = s.m;
    s = joined_lanes(s, heat.c);
    if (RACE)
        best = best_lane(best, s.m > -INFINITY ? s.m : 0.f, heat.c);
    if ((threadIdx.x & 31) == 0) {
        part[threadIdx.x >> 5] = s;
        part_best[threadIdx.x >> 5] = best;
    }
    if (threadIdx.x == 0)
        place = INT_MAX;
    __syncthreads();
    if (heat.greedy) {
        // Whoever has the CTA's maximum looks for its place in its own loads, once more.  (Every
        // thread for its own maximum as it comes by cost all rows: 64 x 5 of 151936 35.4 us, not 34.9.)
        float top = part[0].m;
        for (int w = 1; w < WARPS; ++w)
            top = fmaxf(top, part[w].m);
        if (m == top && m > -INFINITY) {
            int at = INT_MAX;
            if (odd && logit<F32>(p.logits, begin + odd_at) == m)
                at = odd_at;
            constexpr int M = RACE ? G : U;
            uint4 mine[M];
#pragma unroll
            for (int i = 0; i < M; ++i) {
                const int v = (batch + a) / W + i * THREADS;
                mine[i] = v >= lo && v < hi ? __ldg(l + v) : make_uint4(none, none, none, none);
            }
#pragma unroll
            for (int i = 0; i < M; ++i) {
                float x[W];
                spread<F32>(mine[i], x);
#pragma unroll
                for (int j = 0; j < W; ++j)
                    if (x[j] == m)
                        at = min(at, batch + i * THREADS * W + j);
            }
            atomicMin(&place, at);
        }
        __syncthreads();
    }
    if (RACE && threadIdx.x < 32) {
        best = threadIdx.x < WARPS ? part_best[threadIdx.x] : Runner{-INFINITY, 0.f, -1};
        best = best_lane(best, s.m > -INFINITY ? s.m : 0.f, heat.c);
    }
    if (threadIdx.x == 0) {
        for (int w = 1; w < WARPS; ++w)
            s = joined(s, part[w], heat.c);
        int at = heat.greedy && s.m > -INFINITY ? place : -1;
        if (RACE) {
            p.best[(int64_t)seq * p.parts1 + cut] = make_float2(best.x, best.log_e);
            at = heat.greedy ? at : best.at;
        }
        p.stats[(int64_t)row * p.parts1 + cut] = make_float4(s.m, s.z, __int_as_float(at), 0.f);
    }
}

// What is left of a row of probabilities, against e: the best (p - q) / e.
struct Race {
    float m, c, inv_z;
    Pick best;

    // N elements from index v on
    template <int N>
    __device__ __forceinline__ void run(int v, const float (&x)[N], const float (&q)[N], const float (&e)[N])
    {
        float score[N], top = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            float inv;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(e[j]));
            score[j] = fmaf(exp2_of((x[j] - m) * c), inv_z, -q[j]) * inv;
            top = fmaxf(top, score[j]);
        }
        if (top > best.score) {
            best.score = top;
#pragma unroll
            for (int j = N - 1; j >= 0; --j)
                if (score[j] == top)
                    best.at = v + j;
        }
    }
};

// How a row is gone over in the second launch, 8 elements at a time: chunk ch begins at
// element 8 ch - off, on 16 bytes of e.  VEC: logits and q lie alike, and the chunks are the
// row.  Else they are shifted by dl and dq elements, their loads take a neighbour more, and
// the chunks first .. first + count - 1 are those whose loads lie within the row, which leaves
// `head` elements before and `tail` behind them.
struct Walk {
    int off, dl, dq, first, count, head, tail;
};
template <bool F32, bool VEC>
__device__ __forceinline__ Walk walk_of(int vocab, int64_t noise, int64_t logits, int64_t probs)
{
    if (VEC)
        return {0, 0, 0, 0, vocab / 8, 0, 0};
    Walk w;
    w.off = (int)(noise & 3);
    w.dl = (int)(logits - w.off) & (F32 ? 3 : 7);
    w.dq = (int)(probs - w.off) & 3;
    w.first = w.off ? 2 : 1;
    // the last chunk ends at least 8 elements before the row does
    const int behind = vocab - 16 + w.off >= 0 ? (vocab - 16 + w.off) / 8 + 1 : 0;
    w.count = max(behind - w.first, 0);
    w.head = w.count ? 8 * w.first - w.off : vocab;
    w.tail = w.count ? vocab - (8 * behind - w.off) : 0;
    return w;
}

// A chunk's loads of the row, of e and of q.
template <bool F32, bool VEC>
struct Chunk {
    uint4 l[(F32 ? 2 : 1) + !VEC];
    float4 e[2], q[2 + !VEC];
};
template <bool F32, bool VEC>
__device__ __forceinline__ void load_noise(Chunk<F32, VEC> &k, const float *e, const Walk &w, int ch, bool on)
{
#pragma unroll
    for (int j = 0; j < 2; ++j)
        k.e[j] = on ? __ldg(reinterpret_cast<const float4 *>(e - w.off) + 2 * ch + j) : make_float4(1.f, 1.f, 1.f, 1.f);
}
template <bool F32, bool VEC>
__device__ __forceinline__ void load_chunk(Chunk<F32, VEC> &k, const uint8_t *l, const float *q, const Walk &w, int ch, bool on)
{
    constexpr int N = F32 ? 2 : 1, BYTES = F32 ? 4 : 2;
    const uint32_t none = F32 ? 0xFF800000u : 0xFF80FF80u;
#pragma unroll
    for (int j = 0; j < N + !VEC; ++j)
        k.l[j] = on && (j < N || w.dl) ? __ldg(reinterpret_cast<const uint4 *>(l - BYTES * (w.off + w.dl)) + N * ch + j)
                                       : make_uint4(none, none, none, none);
#pragma unroll
    for (int j = 0; j < 2 + !VEC; ++j)
        k.q[j] = on && q != nullptr && (j < 2 || w.dq) ? __ldg(reinterpret_cast<const float4 *>(q - (w.off + w.dq)) + 2 * ch + j)
                                                       : make_float4(0.f, 0.f, 0.f, 0.f);
}
template <int N>
__device__ __forceinline__ void place(float (&x)[4 * N], const float4 (&r)[N], int)
{
#pragma unroll
    for (int j = 0; j < N; ++j)
        x[4 * j] = r[j].x, x[4 * j + 1] = r[j].y, x[4 * j + 2] = r[j].z, x[4 * j + 3] = r[j].w;
}
template <int N>
__device__ __forceinline__ void place(float (&x)[4 * N], const float4 (&r)[N + 1], int d)
{
    shifted<4 * N>(r, d, x);
}
// The chunk's logits, cleaned.
template <bool F32, bool VEC>
__device__ __forceinline__ void place_logits(float (&x)[8], const Chunk<F32, VEC> &k, const Walk &w)
{
    if constexpr (F32) {
        float4 r[2 + !VEC];
#pragma unroll
        for (int j = 0; j < 2 + !VEC; ++j)
            r[j] = make_float4(__uint_as_float(k.l[j].x), __uint_as_float(k.l[j].y), __uint_as_float(k.l[j].z), __uint_as_float(k.l[j].w));
        place<2>(x, r, w.dl);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            x[j] = clean<true>(x[j]);
    } else if constexpr (VEC) {
        spread<false>(k.l[0], x);
    } else {
        spread<false>(shifted(k.l[0], k.l[1], w.dl), x);
    }
}

// What is written of a sequence, by one warp.  s: the sums of the row after its taken drafts.
template <bool F32>
__device__ __forceinline__ void write_result(const VerifyArgs &p, const Stat &s, const Heat &heat, int seq, int taken, int token,
                                             const float *draft_logprob)
{
    const int lane = threadIdx.x & 31, drafts = p.queries - 1;
    const int64_t row = (int64_t)seq * p.queries + taken;
    const float logprob = token < 0 ? 0.f : (logit<F32>(p.logits, row * p.stride + token) - s.m) * heat.c * LN2 - logf(s.z);
    for (int i = lane; i < p.queries; i += 32) {
        const int64_t at = (int64_t)seq * p.queries + i;
        p.tokens[at] = i < taken ? __ldg(p.drafts + (int64_t)seq * drafts + i) : (i == taken ? token : -1);
        if (p.logprobs != nullptr)
            p.logprobs[at] = i < taken ? draft_logprob[i] : (i == taken ? logprob : 0.f);
    }
    if (lane == 0)
        p.accepted[seq] = taken;
}

// The best of chunks lo .. hi - 1 of a row, and with `ends` of its ragged ends, for every
// thread of the CTA.  q: the drafts' probabilities or null; out: an index that is left out,
// or -1.  next: this thread's first noise, loaded already.
template <bool F32, bool VEC>
__device__ Pick row_race(const VerifyArgs &p, const Stat &s, const Heat &heat, int64_t row, const float *e, const float *q, const Walk &w,
                         int out, int lo, int hi, bool ends, Chunk<F32, VEC> &next, Pick (&part)[WARPS])
{
    Race r = {s.m, heat.c, 1.f / s.z, {0.f, -1}};
    const uint8_t *l = static_cast<const uint8_t *>(p.logits) + row * p.stride * (F32 ? 4 : 2);
    load_chunk<F32, VEC>(next, l, q, w, lo + threadIdx.x, lo + (int)threadIdx.x < hi);
    int end_at = -1;
    float end_x = -INFINITY, end_q = 0.f, end_e = 1.f;
    if (!VEC && ends && (int)threadIdx.x < w.head + w.tail) {
        const int t = threadIdx.x;
        end_at = t < w.head ? t : p.vocab - w.tail + t - w.head;
        end_x = end_at == out ? -INFINITY : logit<F32>(p.logits, row * p.stride + end_at);
        end_q = q != nullptr ? __ldg(q + end_at) : 0.f;
        end_e = __ldg(e + end_at);
    }
    for (int ch = lo + threadIdx.x; ch < hi; ch += THREADS) {
        const Chunk<F32, VEC> k = next;
        load_noise<F32, VEC>(next, e, w, ch + THREADS, ch + THREADS < hi);
        load_chunk<F32, VEC>(next, l, q, w, ch + THREADS, ch + THREADS < hi);
        float x[8], ev[8], qv[8];
        place_logits<F32, VEC>(x, k, w);
        place<2>(ev, k.e, 0);
        place<2>(qv, k.q, w.dq);
        const int v = 8 * ch - w.off;
        if (out >= v && out < v + 8)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                x[j] = out == v + j ? -INFINITY : x[j];
        r.run<8>(v, x, qv, ev);
    }
    if (!VEC && end_at >= 0) {
        const float x[1] = {end_x}, qv[1] = {end_q}, ev[1] = {end_e};
        const Pick before = r.best;
        r.best = {0.f, -1};
        r.run<1>(end_at, x, qv, ev);
        r.best = better(before, r.best);
    }
    Pick best = best_lane(r.best);
    __syncthreads();  // part may hold an earlier result
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = best;
    __syncthreads();
    for (int w = 0; w < WARPS; ++w)
        best = better(best, part[w]);
    return best;
}

template <bool F32, bool VEC>
__global__ void __launch_bounds__(THREADS, PICK_CTAS) verify_pick_kernel(const VerifyArgs p)
{
    __shared__ Stat row_stat[MAX_QUERIES];
    __shared__ float draft_logprob[MAX_QUERIES];
    __shared__ int good[MAX_QUERIES];
    __shared__ Pick part[WARPS];
    __shared__ bool last;
    const int seq = blockIdx.x / p.parts2, cut = blockIdx.x % p.parts2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, drafts = p.queries - 1;
    pdl_launch_dependents();
    // The first launch lets this one start only after all that was before it has finished,
    // so what that wrote can be read here; the rows' sums cannot.
    const Heat heat = heat_of(p, seq);
    const int count = count_of(p, seq);
    const float *e = p.noise + (int64_t)seq * p.vocab;
    Walk w = walk_of<F32, VEC>(p.vocab, (int64_t)seq * p.vocab, 0, 0);
    const int lo = w.first + (int)((int64_t)cut * w.count / p.parts2), hi = w.first + (int)((int64_t)(cut + 1) * w.count / p.parts2);
    Chunk<F32, VEC> next;
    if (!p.raced)
        load_noise<F32, VEC>(next, e, w, lo + threadIdx.x, lo + (int)threadIdx.x < hi);
    // a warp's rows are warp, warp + 8, ...: lane i has what draft i of them needs
    const int mine = warp + WARPS * lane;
    int draft = -1;
    float draft_logit = -INFINITY, draft_q = 1.f, draft_u = 0.f;
    if (mine < count) {
        draft = __ldg(p.drafts + (int64_t)seq * drafts + mine);
        if (p.uniforms != nullptr)
            draft_u = __ldg(p.uniforms + (int64_t)seq * drafts + mine);
        if (draft >= 0 && draft < p.vocab) {
            draft_logit = logit<F32>(p.logits, ((int64_t)seq * p.queries + mine) * p.stride + draft);
            if (p.probs != nullptr)
                draft_q = __ldg(p.probs + ((int64_t)seq * drafts + mine) * p.vocab + draft);
        } else {
            draft = -1;
        }
    }
    pdl_wait();
    // the rows' sums, and which drafts hold
    for (int i = warp, j = 0; i <= count; i += WARPS, ++j) {
        const int64_t row = (int64_t)seq * p.queries + i;
        Sum sum = {-INFINITY, 0.f};
        int at = -1;
        if (lane < p.parts1) {
            const float4 v = __ldcg(p.stats + row * p.parts1 + lane);
            sum = {v.x, v.y};
            at = __float_as_int(v.z);
        }
        const float m = sum.m;
        sum = joined_lanes(sum, heat.c);
        const Stat s = {sum.m, sum.z, (int)__reduce_min_sync(0xffffffffu, m == sum.m ? (unsigned)at : UINT_MAX)};
        if (lane == j) {
            row_stat[i] = s;
            int ok = 0;
            if (draft >= 0 && s.z > 0.f) {
                const float x = (draft_logit - s.m) * heat.c;
                ok = heat.greedy ? draft == s.at : draft_u * draft_q < exp2_of(x) / s.z;
                draft_logprob[i] = x * LN2 - logf(s.z);
            }
            good[i] = ok;
        }
    }
    __syncthreads();
    int taken = 0;
    while (taken < count && good[taken])
        ++taken;
    const Stat s = row_stat[taken];
    const int64_t row = (int64_t)seq * p.queries + taken;
    int token = heat.greedy ? s.at : -1;
    const bool race = !heat.greedy && s.z > 0.f;  // else there is nothing to draw, or nothing to draw from
    const bool rest = taken < count;              // a draft was rejected here
    if (race && p.raced) {
        Runner best = {-INFINITY, 0.f, -1};
        if (lane < p.parts1) {
            const float2 v = __ldcg(p.best + (int64_t)seq * p.parts1 + lane);
            best = {v.x, v.y, __float_as_int(__ldcg(p.stats + row * p.parts1 + lane).z)};
        }
        token = best_lane(best, s.m, heat.c).at;
    } else if (race) {
        const int64_t q_row = ((int64_t)seq * drafts + taken) * p.vocab;
        const float *q = rest && p.probs != nullptr ? p.probs + q_row : nullptr;
        w = walk_of<F32, VEC>(p.vocab, (int64_t)seq * p.vocab, row * p.stride, q_row);
        const int out = rest && q == nullptr ? __ldg(p.drafts + (int64_t)seq * drafts + taken) : -1;
        const Pick mine = row_race<F32, VEC>(p, s, heat, row, e, q, w, out, lo, hi, cut == 0, next, part);
        if (threadIdx.x == 0) {
            p.best[(int64_t)seq * p.parts2 + cut] = make_float2(mine.score, __int_as_float(mine.at));
            last = atomic_add_acq_rel(p.arrived + seq, 1u) == (unsigned)p.parts2 - 1;
        }
        __syncthreads();
        if (!last)
            return;
        Pick best = {0.f, -1};
        if (lane < p.parts2) {
            const float2 v = __ldcg(p.best + (int64_t)seq * p.parts2 + lane);
            best = {v.x, __float_as_int(v.y)};
        }
        best = best_lane(best);
        if (best.at < 0 && rest) {  // nothing is left: the drafts' probabilities cover the row, which is drawn from whole
            load_noise<F32, VEC>(next, e, w, w.first + threadIdx.x, (int)threadIdx.x < w.count);
            best = row_race<F32, VEC>(p, s, heat, row, e, nullptr, w, -1, w.first, w.first + w.count, true, next, part);
        }
        token = best.at;
    } else if (cut != 0) {
        return;
    }
    if (warp != 0)
        return;
    write_result<F32>(p, s, heat, seq, taken, token, draft_logprob);
}

struct Layout {
    int parts1, parts2;
    size_t best, arrived, total;
};
Layout layout_of(int seqs, int queries, int vocab, int sm_count, bool raced, bool f32)
{
    // Cuts of a row: what the SMs' CTAs have to do one after the other is the least, a CTA
    // counting PART_MIN elements more than it has; the most cuts of each number of waves.
    auto cuts = [&](int rows, int slots) {
        const int most = vocab / 1024 < 1 ? 1 : (vocab / 1024 < MAX_PARTS ? vocab / 1024 : MAX_PARTS);
        int best = 1;
        int64_t least = INT64_MAX;
        for (int waves = (rows + slots - 1) / slots, tried = 0; tried < 8; ++tried, ++waves) {
            const int n = (int)((int64_t)slots * waves / rows < most ? (int64_t)slots * waves / rows : most);
            const int64_t cost = waves * (int64_t)((vocab + n - 1) / n + PART_MIN);
            if (cost < least) {
                least = cost;
                best = n;
            }
            if (n == most)
                break;
        }
        return best;
    };
    Layout l;
    l.parts1 = cuts(seqs * queries, (raced ? race_ctas(f32) : rows_ctas(f32)) * sm_count);
    l.parts2 = raced ? 1 : cuts(seqs, PICK_CTAS * sm_count);
    size_t o = (size_t)seqs * queries * l.parts1 * sizeof(float4);
    l.best = o;
    o += (size_t)seqs * (raced ? l.parts1 : l.parts2) * sizeof(float2);
    l.arrived = o;
    o += (size_t)seqs * sizeof(unsigned);
    l.total = o;
    return l;
}

template <bool F32, bool VEC>
cudaError_t launch_kind(const VerifyArgs &p, cudaStream_t stream)
{
    const dim3 grid((unsigned)(p.seqs * p.queries * p.parts1));
    // rows of e lie in their loads as the logits' do
    const bool alike = (p.stride - p.vocab) % (F32 ? 4 : 8) == 0;
    const cudaError_t e = !p.raced ? launch_pdl(verify_rows_kernel<F32, NO_RACE>, grid, dim3(THREADS), 0, stream, p)
                          : alike  ? launch_pdl(verify_rows_kernel<F32, RACE_ALIGNED>, grid, dim3(THREADS), 0, stream, p)
                                   : launch_pdl(verify_rows_kernel<F32, RACE_SHIFTED>, grid, dim3(THREADS), 0, stream, p);
    if (e != cudaSuccess)
        return e;
    return launch_pdl(verify_pick_kernel<F32, VEC>, dim3((unsigned)(p.seqs * p.parts2)), dim3(THREADS), 0, stream, p);
}

}  // namespace

size_t verify_workspace(int seqs, int queries, int vocab, int sm_count)
{
    const size_t a = layout_of(seqs, queries, vocab, sm_count, queries == 1, false).total;
    const size_t b = layout_of(seqs, queries, vocab, sm_count, queries == 1, true).total;
    return a > b ? a : b;
}

cudaError_t launch_verify(const Verify &a, int sm_count, void *workspace, cudaStream_t stream)
{
    // rows of logits, q and e that all begin on 16 bytes
    const bool vec = a.vocab % 8 == 0 && a.stride % 8 == 0, raced = a.queries == 1;
    const Layout l = layout_of(a.seqs, a.queries, a.vocab, sm_count, raced, a.f32);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    const VerifyArgs p = {a.logits, a.stride, a.drafts, a.counts, a.probs, a.temperature, a.uniforms, a.noise, a.tokens,
                          a.accepted, a.logprobs, a.seqs, a.queries, a.vocab, l.parts1, l.parts2, raced,
                          reinterpret_cast<float4 *>(ws), reinterpret_cast<float2 *>(ws + l.best),
                          reinterpret_cast<unsigned *>(ws + l.arrived)};
    if (vec)
        return a.f32 ? launch_kind<true, true>(p, stream) : launch_kind<false, true>(p, stream);
    return a.f32 ? launch_kind<true, false>(p, stream) : launch_kind<false, false>(p, stream);
}

}  // namespace w4q
