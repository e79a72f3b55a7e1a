// api_decode.cu -- the extern "C" entry points of w4q.h for the operators
// between the linear layers of a decode step: host-side validation and the
// launches.  Nothing here allocates or synchronizes.
#include "decode.h"
#include "kernels.h"
#include "w4q.h"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int device_sms()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64)
        return -1;
    return w4q::device_sm_count(dev);
}

int status(cudaError_t e) { return e == cudaSuccess ? W4Q_OK : W4Q_ERR_CUDA; }

constexpr int64_t MAX_TOKENS = 1 << 22;
constexpr int MAX_HEADS = 1024, MAX_SEQS = 4096, MAX_ROWS = 64;

bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

// The arguments of a norm and a rotation.
int check_prep(int head_dim, const void *q_weight, const void *k_weight, float eps, const float *cos_sin,
               int64_t positions, int rot)
{
    if (!(eps >= 0.f))
        return W4Q_ERR_INVALID_ARG;
    if (!aligned16(q_weight) || !aligned16(k_weight) || !aligned16(cos_sin))
        return W4Q_ERR_MISALIGNED;
    if (cos_sin != nullptr) {
        if (positions <= 0 || rot <= 0)
            return W4Q_ERR_INVALID_ARG;
        if (rot % 16 != 0 || rot > head_dim)
            return W4Q_ERR_UNSUPPORTED;
    }
    return W4Q_OK;
}

// A row stride holds the row and keeps every row 16-byte aligned.
int check_stride(int64_t stride, int heads, int head_dim)
{
    if (stride < (int64_t)heads * head_dim)
        return W4Q_ERR_INVALID_ARG;
    return stride % 8 == 0 ? W4Q_OK : W4Q_ERR_MISALIGNED;
}

int check_cache(const w4q_kv8_cache *c, w4q::Kv8 *out)
{
    if (c == nullptr || c->k == nullptr || c->v == nullptr || c->k_scale == nullptr || c->v_scale == nullptr ||
        c->block_table == nullptr || c->seq_lens == nullptr)
        return W4Q_ERR_INVALID_ARG;
    if (c->blocks <= 0 || c->seqs <= 0 || c->width <= 0 || c->kv_heads <= 0)
        return W4Q_ERR_INVALID_ARG;
    if (!head_dim_ok(c->head_dim) || c->format < 0 || c->format > 1 || c->seqs > MAX_SEQS ||
        c->kv_heads > MAX_HEADS || c->blocks > 0x7fffffffLL)
        return W4Q_ERR_UNSUPPORTED;
    int log2 = 4;
    while (log2 < 8 && (1 << log2) != c->page)
        ++log2;
    if (log2 == 8)
        return W4Q_ERR_UNSUPPORTED;
    if (((int64_t)c->width << log2) >= 0x7fffffffLL - 127)  // positions are 32-bit
        return W4Q_ERR_UNSUPPORTED;
    if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->k_scale) || !aligned16(c->v_scale) ||
        !aligned16(c->block_table) || !aligned16(c->seq_lens))
        return W4Q_ERR_MISALIGNED;
    *out = w4q::Kv8{static_cast<uint8_t *>(c->k), static_cast<uint8_t *>(c->v), c->k_scale, c->v_scale,
                    c->block_table, c->seq_lens, c->blocks, c->seqs, c->width, c->kv_heads, c->head_dim, log2,
                    c->format == 1};
    return W4Q_OK;
}

int check_moe(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int topk)
{
    if (tokens <= 0 || hidden <= 0 || inter <= 0 || experts <= 0 || topk <= 0 || topk > experts)
        return W4Q_ERR_INVALID_ARG;
    if (tokens > 64 || hidden % 256 != 0 || inter % 256 != 0 || hidden > 32768 || inter > 32768 || experts > 512 ||
        topk > 16 || experts * 2 * inter * hidden > (1LL << 36))  // a packed weight's offsets
        return W4Q_ERR_UNSUPPORTED;
    return W4Q_OK;
}

}  // namespace

extern "C" {

int qk_norm_rope(const void *q, const void *k, int64_t tokens, int q_heads, int k_heads, int head_dim,
                 int64_t q_stride, int64_t k_stride, const void *q_weight, const void *k_weight, float eps,
                 const float *cos_sin, int64_t positions, int rot, int interleaved, const int32_t *pos,
                 void *q_out, void *k_out, void *stream)
{
    if (q == nullptr || q_out == nullptr || tokens < 0 || q_heads <= 0 || k_heads < 0 ||
        (k_heads > 0 && (k == nullptr || k_out == nullptr)))
        return W4Q_ERR_INVALID_ARG;
    if (!head_dim_ok(head_dim) || tokens > MAX_TOKENS || q_heads > MAX_HEADS || k_heads > MAX_HEADS)
        return W4Q_ERR_UNSUPPORTED;
    int st = check_prep(head_dim, q_weight, k_weight, eps, cos_sin, positions, rot);
    if (st == W4Q_OK)
        st = check_stride(q_stride, q_heads, head_dim);
    if (st == W4Q_OK && k_heads > 0)
        st = check_stride(k_stride, k_heads, head_dim);
    if (st != W4Q_OK)
        return st;
    if (!aligned16(q) || !aligned16(k) || !aligned16(q_out) || !aligned16(k_out) || !aligned16(pos))
        return W4Q_ERR_MISALIGNED;
    if (tokens == 0)
        return W4Q_OK;
    const w4q::HeadPrep prep = {q_weight, k_heads > 0 ? k_weight : nullptr, cos_sin, positions,
                                cos_sin ? rot : 0, interleaved != 0, eps};
    return status(w4q::launch_qk_norm_rope(q, k, tokens, q_heads, k_heads, head_dim, q_stride, k_stride, prep, pos,
                                           q_out, k_out, static_cast<cudaStream_t>(stream)));
}

int kv8_append(const w4q_kv8_cache *cache, const void *k, const void *v, int64_t k_stride, int64_t v_stride,
               int64_t tokens, const int32_t *cu_tokens, const void *q, int64_t q_stride, int q_heads, void *q_out,
               const void *q_weight, const void *k_weight, float eps, const float *cos_sin, int64_t positions,
               int rot, int interleaved, void *stream)
{
    w4q::Kv8 c;
    int st = check_cache(cache, &c);
    if (st != W4Q_OK)
        return st;
    if (k == nullptr || v == nullptr || tokens < 0 || q_heads < 0 ||
        (q_heads > 0 && (q == nullptr || q_out == nullptr)) || (cu_tokens == nullptr && tokens != c.seqs))
        return W4Q_ERR_INVALID_ARG;
    if (tokens > MAX_TOKENS || q_heads > MAX_HEADS)
        return W4Q_ERR_UNSUPPORTED;
    st = check_prep(c.head_dim, q_weight, k_weight, eps, cos_sin, positions, rot);
    if (st == W4Q_OK)
        st = check_stride(k_stride, c.kv_heads, c.head_dim);
    if (st == W4Q_OK)
        st = check_stride(v_stride, c.kv_heads, c.head_dim);
    if (st == W4Q_OK && q_heads > 0)
        st = check_stride(q_stride, q_heads, c.head_dim);
    if (st != W4Q_OK)
        return st;
    if (!aligned16(k) || !aligned16(v) || !aligned16(cu_tokens) || (q_heads > 0 && (!aligned16(q) || !aligned16(q_out))))
        return W4Q_ERR_MISALIGNED;
    if (tokens == 0)
        return W4Q_OK;
    const w4q::HeadPrep prep = {q_weight, k_weight, cos_sin, positions, cos_sin ? rot : 0, interleaved != 0, eps};
    return status(w4q::launch_kv8_append(c, k, v, k_stride, v_stride, tokens, cu_tokens, q, q_stride, q_heads, q_out,
                                         prep, static_cast<cudaStream_t>(stream)));
}

int kv8_read(const w4q_kv8_cache *cache, const int32_t *cu_tokens, int64_t tokens, void *k_out, void *v_out,
             void *stream)
{
    w4q::Kv8 c;
    const int st = check_cache(cache, &c);
    if (st != W4Q_OK)
        return st;
    if (k_out == nullptr || v_out == nullptr || tokens < 0 || (cu_tokens == nullptr && tokens != c.seqs))
        return W4Q_ERR_INVALID_ARG;
    if (tokens > MAX_TOKENS)
        return W4Q_ERR_UNSUPPORTED;
    if (!aligned16(cu_tokens) || !aligned16(k_out) || !aligned16(v_out))
        return W4Q_ERR_MISALIGNED;
    if (tokens == 0)
        return W4Q_OK;
    return status(w4q::launch_kv8_read(c, cu_tokens, tokens, k_out, v_out, static_cast<cudaStream_t>(stream)));
}

size_t kv8_workspace_bytes(int64_t seqs, int queries, int heads, int kv_heads, int head_dim)
{
    if (seqs <= 0 || seqs > MAX_SEQS || queries <= 0 || kv_heads <= 0 || heads <= 0 || heads % kv_heads != 0 ||
        kv_heads > MAX_HEADS || queries > MAX_ROWS || (int64_t)queries * (heads / kv_heads) > MAX_ROWS ||
        !head_dim_ok(head_dim))
        return 0;
    const int sms = device_sms();
    return sms < 0 ? 0 : w4q::kv8_attention_workspace(queries, heads / kv_heads, head_dim, sms);
}

int kv8_attention(const w4q_kv8_cache *cache, const void *q, int64_t q_stride, void *out, float *lse, int queries,
                  int heads, float scale, int64_t window, void *workspace, size_t workspace_bytes, void *stream)
{
    w4q::Kv8 c;
    int st = check_cache(cache, &c);
    if (st != W4Q_OK)
        return st;
    if (q == nullptr || out == nullptr || queries <= 0 || heads <= 0 || window < 0 || !(scale == scale))
        return W4Q_ERR_INVALID_ARG;
    if (heads % c.kv_heads != 0 || queries > MAX_ROWS || (int64_t)queries * (heads / c.kv_heads) > MAX_ROWS)
        return W4Q_ERR_UNSUPPORTED;
    // the pieces of 64 positions of all (sequence, kv head, 8 query rows), and their beginnings, are
    // counted in 32 bits
    const int64_t tiles = ((int64_t)queries * (heads / c.kv_heads) + 7) / 8;
    if ((((int64_t)c.width << c.page_log2) / 64 + 8) * c.seqs * c.kv_heads * tiles >= 0x7fffffffLL)
        return W4Q_ERR_UNSUPPORTED;
    st = check_stride(q_stride, heads, c.head_dim);
    if (st != W4Q_OK)
        return st;
    if (!aligned16(q) || !aligned16(out) || !aligned16(lse) || !aligned16(workspace))
        return W4Q_ERR_MISALIGNED;
    const int sms = device_sms();
    if (sms < 0)
        return W4Q_ERR_CUDA;
    if (workspace == nullptr ||
        workspace_bytes < w4q::kv8_attention_workspace(queries, heads / c.kv_heads, c.head_dim, sms))
        return W4Q_ERR_WORKSPACE;
    // a window as long as the table's positions hides nothing
    const int win = window >= ((int64_t)c.width << c.page_log2) ? 0 : (int)window;
    return status(w4q::launch_kv8_attention(c, q, q_stride, out, lse, queries, heads, scale, win, sms, workspace,
                                            static_cast<cudaStream_t>(stream)));
}

size_t moe_workspace_bytes(int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int topk)
{
    if (check_moe(tokens, hidden, inter, experts, topk) != W4Q_OK)
        return 0;
    return w4q::moe_workspace((int)tokens, (int)hidden, (int)inter, topk);
}

int moe_w4a16(const void *x, const void *router, const float *bias, const void *w13, const void *w2, void *out,
              int64_t tokens, int64_t hidden, int64_t inter, int64_t experts, int topk, int sigmoid, int renormalize,
              float scale, int32_t *ids_out, float *weights_out, void *workspace, size_t workspace_bytes, void *stream)
{
    if (x == nullptr || router == nullptr || w13 == nullptr || w2 == nullptr || out == nullptr || !(scale == scale))
        return W4Q_ERR_INVALID_ARG;
    const int st = check_moe(tokens, hidden, inter, experts, topk);
    if (st != W4Q_OK)
        return st;
    if (bias != nullptr && !sigmoid)
        return W4Q_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(router) || !aligned16(bias) || !aligned16(w13) || !aligned16(w2) ||
        !aligned16(out) || !aligned16(ids_out) || !aligned16(weights_out) || !aligned16(workspace))
        return W4Q_ERR_MISALIGNED;
    if (workspace == nullptr || workspace_bytes < w4q::moe_workspace((int)tokens, (int)hidden, (int)inter, topk))
        return W4Q_ERR_WORKSPACE;
    const int sms = device_sms();
    if (sms < 1)
        return W4Q_ERR_CUDA;
    const w4q::Moe a = {x, router, bias, w13, w2, out, ids_out, weights_out, (int)tokens, (int)hidden, (int)inter,
                        (int)experts, topk, sigmoid != 0, renormalize != 0, scale};
    return status(w4q::launch_moe(a, sms, workspace, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
