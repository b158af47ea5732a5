// Internal launcher interface of the language-model operators (linear
// attention with a decay for each head, RMS norm with the residual's addition,
// clipping by the global gradient norm, the gated linear recurrence, the norm of
// queries and keys, the embedding) between mgs_api.cu and the kernels.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mgscan.h"
#include "mgs_device.cuh"

namespace mgs {

constexpr int64_t kAttnChunk = 128;   // time steps of a chunk; segments are whole chunks

// One walk over time of out_t = o_scale * S_t^T q_t with
//   forward:  S_t = e^{g_t} S_{t-1} + kv_scale * k_t v_t^T,  t = 0..T-1
//   reverse:  S_t = S'_{t+1} + kv_scale * k_t v_t^T, S'_t = e^{g_t} S_t,  t = T-1..0
// where q, k, v stand for whichever tensors have those roles (attention
// itself and each of its three gradients are one walk).  Strides are
// (batch, time, head) in elements; head h of the walk reads head h / div.
struct AttnWalk {
    const void *q, *k, *v;
    const void *x;                // partner of row_dot (null: none)
    int64_t qs[3], ks[3], vs[3], xs[3], os[3];
    int qdiv, kdiv, vdiv, xdiv;
    void *out;                    // null: only the state is wanted
    int out_f32;                  // out is fp32 whatever the inputs' type
    const float *s_in;            // state at the walk's start, [B H][D][D] (null: zeros)
    int s_in_t;                   // ... stored transposed
    float *s_out;                 // state at the walk's end, [B H][D][D] (null: not wanted)
    float *row_dot;               // [parts][B H][T]: <out_t, x_t> before rounding, in parts to be added
    float *ckpt;                  // [B H][spans][D][D]: the state at the first `kept` spans' ends (null: not wanted)
    const float *seg_in;          // [B H][nseg][D][D]: the state at each segment's start (nseg > 1)
    float *seg_out;               // [B H][nseg][D][D]: state-only pass: each segment's own state
    float o_scale, kv_scale;
    int rev;
};

struct AttnSet {
    AttnWalk w[3];
    const float *g;
    int64_t gs[3];
    int64_t B, T, H;
    int first;                    // the launch's first walk
    int beside;                   // launched beside other walks, with whose kernel it shares nothing but its end
    int64_t seg_len;              // steps of a segment (a multiple of kAttnChunk)
    int nseg, spans, kept;
    int span;                     // steps between two states that are kept: whole chunks
    uint32_t tries;               // a barrier wait's limit: tries of about 40 ns
    DevCtl ctl;
};

// Kernels of one call that follow one another: the next one's blocks are set up
// while the last of this one's still run (griddep_launch, called by a block, lets
// them be launched when all blocks have called it), and wait for what this one
// writes (griddep_wait: until it has ended).
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_next(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s, bool early,
                        A... args) {
    cudaLaunchConfig_t c = {};
    c.gridDim = grid, c.blockDim = dim3(threads), c.dynamicSmemBytes = smem, c.stream = s;
    cudaLaunchAttribute a = {};
    a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    a.val.programmaticStreamSerializationAllowed = 1;
    c.attrs = &a, c.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// SIMT walk: the recurrence itself in fp32, any supported type and size
cudaError_t launch_attn_rec(const AttnSet &set, int nwalks, int D, int dtype, bool state_only, cudaStream_t s);

// Tensor-core walks `first` .. of the set.  terms: bf16 terms of the computed
// operands of the output.  fp32: q, k and v are each three dense
// bf16 tensors behind one another (attn_split), out and x are fp32.
// early: it follows a kernel of the same call that lets it be launched early;
// beside: that kernel is of other walks, beside which these run.
cudaError_t launch_attn_mma(const AttnSet &set, int first, int nwalks, int D, int dtype, int terms, bool state_only,
                            bool early, bool beside, cudaStream_t s);

size_t attn_workspace_bytes(const mgs_attention_shape &sh, bool backward);
cudaError_t launch_attn_fwd(const mgs_attention_shape &sh, const void *q, const void *k, const void *v,
                            const float *g, const float *S0, void *o, float *ST, void *ws, const DevCtl &ctl,
                            cudaStream_t s);
cudaError_t launch_attn_bwd(const mgs_attention_shape &sh, const void *q, const void *k, const void *v,
                            const float *g, const float *S0, const void *go, const float *gST, void *dq, void *dk,
                            void *dv, float *dg, float *dS0, void *ws, const DevCtl &ctl, cudaStream_t s);
cudaError_t launch_attn_step(const mgs_attention_shape &sh, const void *q, const void *k, const void *v,
                             const float *g, float *S, const int32_t *slots, int64_t nslots, void *o,
                             cudaStream_t s);

cudaError_t launch_rms_norm_fwd(int dtype, const void *x, const void *res, const void *w, float eps, void *r, void *y,
                                float *rstd, int64_t rows, int64_t N, cudaStream_t s);
cudaError_t launch_rms_norm_fp8(int dtype, const void *x, const void *res, const void *w, float eps, void *r,
                                void *q8, float *scales, int64_t rows, int64_t N, int group, cudaStream_t s);
size_t rms_norm_bwd_workspace_bytes(int64_t rows, int64_t N);
cudaError_t launch_rms_norm_bwd(int dtype, const void *r, const void *w, const float *rstd, const void *gy,
                                const void *gr, void *dx, void *dw, int64_t rows, int64_t N, void *ws,
                                cudaStream_t s);

size_t clip_workspace_bytes(int64_t count);
cudaError_t launch_clip(const void *const *in, void *const *out, const int64_t *numel, const int32_t *dtypes,
                        int64_t count, float max_norm, float *norm, void *ws, cudaStream_t s);

cudaError_t launch_gated_fwd(const mgs_gated_shape &sh, const void *gate, const void *value, const float *h0, void *h,
                             float *hT, float *carries, const DevCtl &ctl, cudaStream_t s);
cudaError_t launch_gated_bwd(const mgs_gated_shape &sh, const void *gate, const void *value, const float *carries,
                             const void *gh, const float *ghT, void *dgate, void *dvalue, float *dh0,
                             const DevCtl &ctl, cudaStream_t s);
cudaError_t launch_gated_step(const mgs_gated_shape &sh, const void *gate, const void *value, float *state,
                              const int32_t *slots, int64_t nslots, void *h, cudaStream_t s);
// late_ns: how late a block comes to a round (of no effect with a late_block that is none)
cudaError_t launch_exchange_check(int late_block, int late_round, uint64_t late_ns, int32_t *rounds, int32_t *wrong,
                                  const DevCtl &ctl, cudaStream_t s);

cudaError_t launch_qk_norm_fwd(const mgs_qk_norm_shape &sh, const void *q, const void *k, const void *qw,
                               const void *kw, const float *table, const int32_t *positions, void *yq, void *yk,
                               cudaStream_t s);
size_t qk_norm_bwd_workspace_bytes(const mgs_qk_norm_shape &sh);
cudaError_t launch_qk_norm_bwd(const mgs_qk_norm_shape &sh, const void *q, const void *k, const void *qw,
                               const void *kw, const void *gq, const void *gk, const float *table,
                               const int32_t *positions, void *dq, void *dk, void *dqw, void *dkw, void *ws,
                               cudaStream_t s);

cudaError_t launch_embed_fwd(int itype, int dtype, const void *tokens, const void *w, float scale, void *out,
                             int64_t N, int64_t V, int64_t D, cudaStream_t s);
size_t embed_bwd_workspace_bytes(int64_t N, int64_t V, int64_t D);
cudaError_t launch_embed_bwd(int itype, int dtype, const void *tokens, const void *grad, int64_t gs, float scale,
                             void *dw, int64_t N, int64_t V, int64_t D, void *ws, cudaStream_t s);

}  // namespace mgs
