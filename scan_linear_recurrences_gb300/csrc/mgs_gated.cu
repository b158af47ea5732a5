// The gated linear recurrence (minGRU) from its pre-activations.  Per channel, with
// z = sigmoid(gate) and c = value, or c = g(value) where g(v) = v + 1/2 for v >= 0,
// sigmoid(v) below,
//   h_t = (1 - z_t) h_{t-1} + z_t c_t.
// Backward, with a = 1 - z = sigmoid(-gate) and L_t = dL/dh_t = gh_t + a_{t+1} L_{t+1}:
//   dvalue = L z c',  dgate = L (c - h_{t-1}) z a,  dh0 = a_1 L_1.
#include "mgs_lm.h"
#include "mgs_num.cuh"

namespace mgs {
namespace {

constexpr int kSpan = MGS_GATED_SPAN;  // steps between two states that the forward keeps for the backward

// z, a = 1 - z, c and c' of one element; both z and a to their own last digits.  A
// gate of -infinity masks the step: c is not looked at.
template <bool POS>
__device__ __forceinline__ void gates(float k, float v, float &z, float &a, float &c, float &slope) {
    const float e = expf(-fabsf(k)), r = 1.f / (1.f + e), er = e * r;
    z = k >= 0.f ? r : er;
    a = k >= 0.f ? er : r;
    if (k != k) z = a = k;
    c = v, slope = 1.f;
    if (POS) {
        const float f = expf(-fabsf(v)), s = 1.f / (1.f + f), fs = f * s;
        c = v < 0.f ? fs : v + 0.5f;
        slope = v < 0.f ? s * fs : 1.f;
    }
    if (k == -INFINITY) c = 0.f, slope = 0.f;
}

template <typename T, bool POS>
__global__ void gated_fwd_kernel(const T *gate, const T *value, const float *h0, T *h, float *hT, float *carries,
                                 int64_t B, int64_t T_, int64_t D, int64_t kb, int64_t kt, int64_t vb, int64_t vt) {
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x, spans = (T_ + kSpan - 1) / kSpan;
    if (i >= B * D) return;
    const int64_t b = i / D, d = i % D;
    float s = h0 ? h0[i] : 0.f;
    for (int64_t t = 0; t < T_; ++t) {
        if (carries && t % kSpan == 0) carries[(b * spans + t / kSpan) * D + d] = s;
        float z, a, c, slope;
        gates<POS>(to_f(gate[b * kb + t * kt + d]), to_f(value[b * vb + t * vt + d]), z, a, c, slope);
        s = fmaf(a, s, z * c);
        h[(b * T_ + t) * D + d] = from_f<T>(s);
    }
    if (hT) hT[i] = s;
}

template <typename T, bool POS>
__global__ void gated_bwd_kernel(const T *gate, const T *value, const float *carries, const T *gh, const float *ghT,
                                 T *dgate, T *dvalue, float *dh0, int64_t B, int64_t T_, int64_t D, int64_t kb,
                                 int64_t kt, int64_t vb, int64_t vt, int64_t gb, int64_t gt) {
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x, spans = (T_ + kSpan - 1) / kSpan;
    if (i >= B * D) return;
    const int64_t b = i / D, d = i % D;
    float flow = ghT ? ghT[i] : 0.f;
    for (int64_t n = spans - 1; n >= 0; --n) {
        float before[kSpan], s = carries[(b * spans + n) * D + d], z, a, c, slope;
        const int len = int(min64(kSpan, T_ - n * kSpan));
        for (int j = 0; j < len; ++j) {
            const int64_t t = n * kSpan + j;
            before[j] = s;
            gates<POS>(to_f(gate[b * kb + t * kt + d]), to_f(value[b * vb + t * vt + d]), z, a, c, slope);
            s = fmaf(a, s, z * c);
        }
        for (int j = len - 1; j >= 0; --j) {
            const int64_t t = n * kSpan + j;
            gates<POS>(to_f(gate[b * kb + t * kt + d]), to_f(value[b * vb + t * vt + d]), z, a, c, slope);
            const float lam = flow + to_f(gh[b * gb + t * gt + d]), lz = lam * z;
            dvalue[(b * T_ + t) * D + d] = from_f<T>(lz * slope);
            dgate[(b * T_ + t) * D + d] = from_f<T>(lz * a * (c - before[j]));
            flow = a * lam;
        }
    }
    if (dh0) dh0[i] = flow;
}

template <typename T, bool POS>
__global__ void gated_step_kernel(const T *gate, const T *value, float *state, const int32_t *slots, int64_t nslots,
                                  T *h, int64_t B, int64_t D, int64_t kb, int64_t vb) {
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= B * D) return;
    const int64_t b = i / D, d = i % D, slot = slots ? slots[b] : b;
    float s = 0.f;
    if (slot >= 0 && slot < nslots) {
        float z, a, c, slope;
        gates<POS>(to_f(gate[b * kb + d]), to_f(value[b * vb + d]), z, a, c, slope);
        s = fmaf(a, state[slot * D + d], z * c);
        state[slot * D + d] = s;
    }
    h[i] = from_f<T>(s);
}

unsigned blocks_of(int64_t n) { return unsigned((n + 127) / 128); }

template <typename T, bool POS>
cudaError_t fwd_go(const mgs_gated_shape &sh, const void *gate, const void *value, const float *h0, void *h, float *hT,
                   float *carries, cudaStream_t s) {
    gated_fwd_kernel<T, POS><<<blocks_of(sh.B * sh.D), 128, 0, s>>>(
        (const T *)gate, (const T *)value, h0, (T *)h, hT, carries, sh.B, sh.T, sh.D, sh.gate_stride[0],
        sh.gate_stride[1], sh.value_stride[0], sh.value_stride[1]);
    return cudaGetLastError();
}
template <typename T, bool POS>
cudaError_t bwd_go(const mgs_gated_shape &sh, const void *gate, const void *value, const float *carries,
                   const void *gh, const float *ghT, void *dgate, void *dvalue, float *dh0, cudaStream_t s) {
    gated_bwd_kernel<T, POS><<<blocks_of(sh.B * sh.D), 128, 0, s>>>(
        (const T *)gate, (const T *)value, carries, (const T *)gh, ghT, (T *)dgate, (T *)dvalue, dh0, sh.B, sh.T, sh.D,
        sh.gate_stride[0], sh.gate_stride[1], sh.value_stride[0], sh.value_stride[1], sh.gh_stride[0],
        sh.gh_stride[1]);
    return cudaGetLastError();
}
template <typename T, bool POS>
cudaError_t step_go(const mgs_gated_shape &sh, const void *gate, const void *value, float *state,
                    const int32_t *slots, int64_t nslots, void *h, cudaStream_t s) {
    gated_step_kernel<T, POS><<<blocks_of(sh.B * sh.D), 128, 0, s>>>((const T *)gate, (const T *)value, state, slots,
                                                                    nslots, (T *)h, sh.B, sh.D, sh.gate_stride[0],
                                                                    sh.value_stride[0]);
    return cudaGetLastError();
}

}  // namespace

#define MGS_BY_TYPE(go, ...)                                                                              \
    (sh.dtype == MGS_BF16 ? (sh.positive ? go<bf16, true>(__VA_ARGS__) : go<bf16, false>(__VA_ARGS__))    \
                          : (sh.positive ? go<float, true>(__VA_ARGS__) : go<float, false>(__VA_ARGS__)))

cudaError_t launch_gated_fwd(const mgs_gated_shape &sh, const void *gate, const void *value, const float *h0, void *h,
                             float *hT, float *carries, cudaStream_t s) {
    return MGS_BY_TYPE(fwd_go, sh, gate, value, h0, h, hT, carries, s);
}
cudaError_t launch_gated_bwd(const mgs_gated_shape &sh, const void *gate, const void *value, const float *carries,
                             const void *gh, const float *ghT, void *dgate, void *dvalue, float *dh0, cudaStream_t s) {
    return MGS_BY_TYPE(bwd_go, sh, gate, value, carries, gh, ghT, dgate, dvalue, dh0, s);
}
cudaError_t launch_gated_step(const mgs_gated_shape &sh, const void *gate, const void *value, float *state,
                              const int32_t *slots, int64_t nslots, void *h, cudaStream_t s) {
    return MGS_BY_TYPE(step_go, sh, gate, value, state, slots, nslots, h, s);
}
#undef MGS_BY_TYPE

}  // namespace mgs
