// decode.h -- host-side launchers of the operators around the linear layer in
// a decode step (internal; the public ABI is w4q.h): head norms with rotation,
// the 8-bit cache's writer, reader and attention, the mixture of experts.
// Every launcher only launches: validation happens in api_decode.cu.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace w4q {

// Launch with programmatic stream serialization, as the library's other
// kernels: the kernel may start while its predecessor finishes and waits
// (griddepcontrol.wait) before it reads or writes global memory.
template <class... KArgs, class... Args>
inline cudaError_t launch_pdl(void (*fn)(KArgs...), dim3 grid, dim3 block, size_t smem,
                              cudaStream_t stream, Args... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, fn, args...);
}

// The paged 8-bit cache (layout in w4q.h).
struct Kv8 {
    uint8_t *k, *v;
    float *k_scale, *v_scale;
    const int32_t *table;
    const int32_t *lens;
    int64_t blocks;
    int seqs, width, kv_heads, head_dim, page_log2;
    bool fp8;
};

// --- attention over the cache (kv8_attention.cu)
size_t kv8_attention_workspace(int queries, int group, int head_dim, int sm_count);
cudaError_t launch_kv8_attention(const Kv8 &c, const void *q, int64_t q_stride, void *out, float *lse,
                                 int queries, int heads, float scale, int window, int sm_count,
                                 void *workspace, cudaStream_t stream);

// --- head norms and rotation, the cache's writer and reader (kv8_append.cu)
struct HeadPrep {
    const void *q_weight, *k_weight;  // bf16 [head_dim] or null: no norm
    const float *cos_sin;             // fp32 [positions][rot] or null: no rotation
    int64_t positions;
    int rot;
    bool interleaved;
    float eps;
};
cudaError_t launch_qk_norm_rope(const void *q, const void *k, int64_t tokens, int q_heads, int k_heads,
                                int head_dim, int64_t q_stride, int64_t k_stride, const HeadPrep &prep,
                                const int32_t *pos, void *q_out, void *k_out, cudaStream_t stream);
cudaError_t launch_kv8_append(const Kv8 &c, const void *k, const void *v, int64_t k_stride,
                              int64_t v_stride, int64_t tokens, const int32_t *cu, const void *q,
                              int64_t q_stride, int q_heads, void *q_out, const HeadPrep &prep,
                              cudaStream_t stream);
cudaError_t launch_kv8_read(const Kv8 &c, const int32_t *cu, int64_t tokens, void *k_out, void *v_out,
                            cudaStream_t stream);

// --- mixture of experts (moe_w4.cu)
struct Moe {
    const void *x, *router;
    const float *bias;
    const void *w13, *w2;
    void *out;
    int32_t *ids_out;
    float *weights_out;
    int tokens, hidden, inter, experts, topk;
    bool sigmoid, renormalize;
    float scale;
};
size_t moe_workspace(int tokens, int hidden, int inter, int topk);
cudaError_t launch_moe(const Moe &a, int sm_count, void *workspace, cudaStream_t stream);

}  // namespace w4q
