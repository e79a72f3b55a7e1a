// rms_norm.cu -- the residual's addition and a root-mean-square norm in one
// pass, into bf16 or into the int8 codes and scales of a W4A8 product.
//
//     s = x + residual;  sum = bf16(s);  y = (s * weight) / sqrt(mean s^2 + eps)
//     bf16:  out = bf16(y)
//     codes: a = max |y| over the row, or over each group of 32;
//            scale = a / 127,  code = rint(y * (1 / scale)) in [-127, 127]
//
// all of it in fp32, each output rounded once (the codes from y itself, not
// from bf16(y), whose rounding would move them by up to a quarter of a step).
// Multiplying the weight in before the root makes the row's scale known with
// the row's sum: rounding is monotonic, so max |y| = max |s * weight| * rstd to
// the bit, and the two reductions share one barrier.
//
// What bounds it: prompts move 8 bytes an element (7 with codes) through HBM;
// a few tokens are one launch's chain of a load, a reduction and a store.
// Layout: a row belongs to the warps of one CTA, a thread holds up to V chunks
// of 8 elements in registers, so every element is read and written once.
#include "common.cuh"
#include "decode.h"

namespace w4q {

namespace {

// Of a CTA, whose kernels then have at most 64 registers: 4 chunks a thread took 72 with 512
// threads, and one CTA an SM from 1024 chunks on (4000 x 16384 into codes 97 us, 72 so).
constexpr int MAX_THREADS = 1024;

struct NormArgs {
    const __nv_bfloat16 *x, *residual, *weight;
    __nv_bfloat16 *sum, *out;
    int8_t *codes;
    float *scales;
    int64_t x_stride, r_stride, sum_stride;
    int tokens, n8;  // n8: chunks of 8 elements of a row
    float eps, inv_hidden;
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 8 elements as pairs.
struct Eight {
    float2 v[4];
};
__device__ __forceinline__ Eight unpack(uint4 r)
{
    return {{{bf16lo_to_f32(r.x), bf16hi_to_f32(r.x)},
             {bf16lo_to_f32(r.y), bf16hi_to_f32(r.y)},
             {bf16lo_to_f32(r.z), bf16hi_to_f32(r.z)},
             {bf16lo_to_f32(r.w), bf16hi_to_f32(r.w)}}};
}
__device__ __forceinline__ uint4 pack8(const Eight &e)
{
    return make_uint4(pack2(e.v[0].x, e.v[0].y), pack2(e.v[1].x, e.v[1].y), pack2(e.v[2].x, e.v[2].y), pack2(e.v[3].x, e.v[3].y));
}

// The larger one; NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float top_of(const Eight &e)
{
    float a = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        a = max_nan(a, max_nan(fabsf(e.v[j].x), fabsf(e.v[j].y)));
    return a;
}

// The codes of y under `scale`: 0 where it is 0, infinite or NaN (the scale then says
// that the values are not finite).  rint(y / scale) as the lowest byte of y * (1 / scale) +
// 1.5 * 2^23, one rounding: the reciprocal's own is 2^-17 of a step, and |y| <= 127 scale
// (1 + 2^-23) needs no clamp.  The activation quantizer rounds the quotient, which gives the
// other code of two where y / scale lies within 2^-16 of their middle, from which both are
// equally far.  (Its rule with quotients everywhere: 3001 x 8192 by groups 39 us, 30.7 so;
// with quotients only where a second product with a reciprocal two bits off gives another
// code: 32.4, without a residual 24.5 instead of 21.9, 700 x 12288 by rows 10.1 instead of 7.0.)
__device__ __forceinline__ uint2 codes_of(const Eight &y, float scale)
{
    uint32_t q[2] = {0u, 0u};
    if (scale >= 0x1p-120f && scale <= 3.4e38f) {
        const float r = __frcp_rn(scale), magic = 12582912.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float2 a = fma2(y.v[2 * h], {r, r}, {magic, magic}), b = fma2(y.v[2 * h + 1], {r, r}, {magic, magic});
            q[h] = prmt(prmt(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040), prmt(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040),
                        0x5410);
        }
    } else if (scale > 0.f && scale < 1.f) {
        // its reciprocal has no room in fp32; and the scale may be far from y / 127
        const float r = __frcp_rn(scale * 0x1p64f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = (j % 2 ? y.v[j / 2].y : y.v[j / 2].x) * 0x1p64f * r;
            q[j / 4] |= ((uint32_t)__float2int_rn(fminf(fmaxf(v, -127.f), 127.f)) & 0xffu) << (8 * (j % 4));
        }
    }
    return make_uint2(q[0], q[1]);
}

// FORM 0: no codes; 1: codes with a scale per row; 2: per group of 32.
// blockDim = (threads of a row, rows); a row's threads are whole warps.
template <int FORM, int V>
__global__ void __launch_bounds__(MAX_THREADS) rms_norm_kernel(const NormArgs p)
{
    __shared__ float part_sum[32];
    __shared__ float part_top[32];
    pdl_launch_dependents();
    const int warps = blockDim.x >> 5, warp = threadIdx.y * warps + (threadIdx.x >> 5);
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < p.tokens;
    pdl_wait();

    // sum may be the residual or x itself: a thread reads all its elements before it writes one
    uint4 xr[V], rr[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        const bool on = live && c < p.n8;
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        xr[i] = on ? *(reinterpret_cast<const uint4 *>(p.x + row * p.x_stride) + c) : zero;
        rr[i] = on && p.residual ? *(reinterpret_cast<const uint4 *>(p.residual + row * p.r_stride) + c) : zero;
    }
    Eight s[V];
    float2 squares = {0.f, 0.f};
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        s[i] = unpack(xr[i]);
        if (p.residual) {
            const Eight r = unpack(rr[i]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[i].v[j] = add2(s[i].v[j], r.v[j]);
            if (p.sum && live && c < p.n8)
                *(reinterpret_cast<uint4 *>(p.sum + row * p.sum_stride) + c) = pack8(s[i]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            squares = fma2(s[i].v[j], s[i].v[j], squares);
        if (p.weight) {
            const Eight w = unpack(c < p.n8 ? __ldg(reinterpret_cast<const uint4 *>(p.weight) + c) : make_uint4(0u, 0u, 0u, 0u));
#pragma unroll
            for (int j = 0; j < 4; ++j)
                s[i].v[j] = mul2(s[i].v[j], w.v[j]);
        }
        if (FORM == 1)
            top = max_nan(top, top_of(s[i]));
    }
    float total = squares.x + squares.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        total += __shfl_xor_sync(0xffffffffu, total, o);
        if (FORM == 1)
            top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
    if (warps > 1) {
        if ((threadIdx.x & 31) == 0) {
            part_sum[warp] = total;
            part_top[warp] = top;
        }
        __syncthreads();
        const int lane = threadIdx.x & 31, at = threadIdx.y * warps + lane;
        total = lane < warps ? part_sum[at] : 0.f;
        top = FORM == 1 && lane < warps ? part_top[at] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            total += __shfl_xor_sync(0xffffffffu, total, o);
            if (FORM == 1)
                top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
        }
    }
    const float rstd = rsqrtf(fmaf(total, p.inv_hidden, p.eps));
    float scale = 0.f;
    if (FORM == 1) {
        scale = __fdiv_rn(top * rstd, 127.f);
        if (live && threadIdx.x == 0)
            p.scales[row] = scale;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = i * blockDim.x + threadIdx.x;
        const bool on = live && c < p.n8;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            s[i].v[j] = mul2(s[i].v[j], {rstd, rstd});
        if (FORM == 2) {
            float a = top_of(s[i]);
            a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 1));
            a = max_nan(a, __shfl_xor_sync(0xffffffffu, a, 2));
            scale = __fdiv_rn(a, 127.f);
            if (on && (c & 3) == 0)
                p.scales[row * (p.n8 >> 2) + (c >> 2)] = scale;
        }
        if (FORM != 0 && on)
            *(reinterpret_cast<uint2 *>(p.codes) + row * p.n8 + c) = codes_of(s[i], scale);
        if (p.out && on)
            *(reinterpret_cast<uint4 *>(p.out) + row * p.n8 + c) = pack8(s[i]);
    }
}

template <int FORM>
cudaError_t launch_form(const NormArgs &p, int v, dim3 grid, dim3 block, cudaStream_t stream)
{
    switch (v) {
    case 1: return launch_pdl(rms_norm_kernel<FORM, 1>, grid, block, 0, stream, p);
    case 2: return launch_pdl(rms_norm_kernel<FORM, 2>, grid, block, 0, stream, p);
    default: return launch_pdl(rms_norm_kernel<FORM, 4>, grid, block, 0, stream, p);
    }
}

// Threads that an SM's 65536 registers hold of these kernels: 28 each with one chunk, 34 with two (40
// are given out), 40 to 42 for codes (48), 56 to 60 with four (64).  (With 1024 for two chunks and 1280
// for codes with one, 1500 x 2048 by groups took 5.5 us, 4.2 so, 700 x 4096 in bf16 4.8, now 4.0, 300 x
// 6656 by rows 3.9, now 3.5; 200 x 16384 in bf16 without a residual 4.1, now 4.8.)
constexpr int at_once(int chunks, bool codes) { return chunks > 2 ? 1024 : (chunks > 1 ? (codes ? 1344 : 1632) : 2048); }

}  // namespace

cudaError_t launch_rms_norm(const Norm &a, int sm_count, cudaStream_t stream)
{
    NormArgs p;
    p.x = static_cast<const __nv_bfloat16 *>(a.x);
    p.residual = static_cast<const __nv_bfloat16 *>(a.residual);
    p.weight = static_cast<const __nv_bfloat16 *>(a.weight);
    p.sum = static_cast<__nv_bfloat16 *>(a.sum_out);
    p.out = static_cast<__nv_bfloat16 *>(a.out);
    p.codes = a.codes;
    p.scales = a.scales;
    p.x_stride = a.x_stride;
    p.r_stride = a.r_stride;
    p.sum_stride = a.sum_stride;
    p.tokens = (int)a.tokens;
    p.n8 = (int)(a.hidden / 8);
    p.eps = a.eps;
    p.inv_hidden = 1.f / (float)a.hidden;
    // The fewest chunks a thread with which all rows run at once, for the shortest chain (into bf16,
    // 1000 x 2048 3.3 us with 1, 3.8 and 4.5 with 2 and 4; 500 x 8192 6.1 with 4, 6.6 with 2).  More
    // rows: two (8191 x 6656 64 us; with 1 and 4 82 and 65; 4000 x 4096 into codes 20.9, 22.5 with
    // 4), four where two make CTAs of many threads (3001 x 8192 into codes 31 us, 33 with 2).
    const bool codes = a.codes != nullptr;
    const int64_t all = a.tokens * p.n8;
    int chunks = 1;
    while (p.n8 > chunks * MAX_THREADS || (chunks < 4 && all > (int64_t)chunks * at_once(chunks, codes) * sm_count))
        chunks *= 2;
    if (all > (int64_t)chunks * at_once(chunks, codes) * sm_count)
        chunks = p.n8 > (codes ? 768 : 1024) ? 4 : 2;
    const int threads = ((p.n8 + chunks - 1) / chunks + 31) / 32 * 32;
    const int rows = threads >= 256 || a.tokens <= sm_count ? 1 : 256 / threads;
    const dim3 grid((unsigned)((a.tokens + rows - 1) / rows)), block((unsigned)threads, (unsigned)rows);
    if (a.codes == nullptr)
        return launch_form<0>(p, chunks, grid, block, stream);
    return a.row_scale ? launch_form<1>(p, chunks, grid, block, stream) : launch_form<2>(p, chunks, grid, block, stream);
}

}  // namespace w4q
