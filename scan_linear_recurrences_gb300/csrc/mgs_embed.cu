// Embedding: out[n] = scale W[token_n], and the table's gradient
// dW[v] = scale * (the sum of grad[n] over the n with token_n = v), in the order of n.
// A token outside 0..V-1 has a row of zeros and no gradient.
#include "mgs_lm.h"
#include "mgs_num.cuh"

namespace mgs {
namespace {

template <typename I, typename T>
__global__ void embed_fwd_kernel(const I *tokens, const T *w, float scale, T *out, int64_t N, int64_t V, int64_t D) {
    for (int64_t n = blockIdx.x; n < N; n += gridDim.x) {
        const int64_t v = int64_t(tokens[n]);
        for (int64_t d = threadIdx.x; d < D; d += blockDim.x)
            out[n * D + d] = from_f<T>(v >= 0 && v < V ? scale * to_f(w[v * D + d]) : 0.f);
    }
}

// a block looks through the tokens for its row
template <typename I, typename T>
__global__ void embed_bwd_kernel(const I *tokens, const T *grad, int64_t gs, float scale, T *dw, int64_t N, int64_t V,
                                 int64_t D) {
    __shared__ int found[256];
    for (int64_t v = blockIdx.x; v < V; v += gridDim.x)
        for (int64_t d0 = 0; d0 < D; d0 += 256) {
            float s = 0.f;
            for (int64_t n0 = 0; n0 < N; n0 += 256) {
                const int64_t n = n0 + threadIdx.x, d = d0 + threadIdx.x;
                const int hit = n < N && int64_t(tokens[n]) == v;
                if (!__syncthreads_or(hit)) continue;
                found[threadIdx.x] = hit;
                __syncthreads();
                for (int i = 0; i < 256; ++i)
                    if (found[i] && d < D) s += to_f(grad[(n0 + i) * gs + d]);
                __syncthreads();
            }
            if (d0 + threadIdx.x < D) dw[v * D + d0 + threadIdx.x] = from_f<T>(scale * s);
        }
}

template <typename I, typename T>
cudaError_t fwd_go(const void *tokens, const void *w, float scale, void *out, int64_t N, int64_t V, int64_t D,
                   cudaStream_t s) {
    embed_fwd_kernel<I, T><<<unsigned(min64(N, 152 * 8)), 256, 0, s>>>((const I *)tokens, (const T *)w, scale,
                                                                      (T *)out, N, V, D);
    return cudaGetLastError();
}
template <typename I, typename T>
cudaError_t bwd_go(const void *tokens, const void *grad, int64_t gs, float scale, void *dw, int64_t N, int64_t V,
                   int64_t D, cudaStream_t s) {
    embed_bwd_kernel<I, T><<<unsigned(min64(V, 152 * 8)), 256, 0, s>>>((const I *)tokens, (const T *)grad, gs, scale,
                                                                      (T *)dw, N, V, D);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_embed_fwd(int itype, int dtype, const void *tokens, const void *w, float scale, void *out,
                             int64_t N, int64_t V, int64_t D, cudaStream_t s) {
    auto *go = itype == MGS_I64 ? (dtype == MGS_BF16 ? fwd_go<int64_t, bf16> : fwd_go<int64_t, float>)
                                : (dtype == MGS_BF16 ? fwd_go<int32_t, bf16> : fwd_go<int32_t, float>);
    return go(tokens, w, scale, out, N, V, D, s);
}

size_t embed_bwd_workspace_bytes(int64_t, int64_t, int64_t) { return 256; }

cudaError_t launch_embed_bwd(int itype, int dtype, const void *tokens, const void *grad, int64_t gs, float scale,
                             void *dw, int64_t N, int64_t V, int64_t D, void *, cudaStream_t s) {
    auto *go = itype == MGS_I64 ? (dtype == MGS_BF16 ? bwd_go<int64_t, bf16> : bwd_go<int64_t, float>)
                                : (dtype == MGS_BF16 ? bwd_go<int32_t, bf16> : bwd_go<int32_t, float>);
    return go(tokens, grad, gs, scale, dw, N, V, D, s);
}

}  // namespace mgs
