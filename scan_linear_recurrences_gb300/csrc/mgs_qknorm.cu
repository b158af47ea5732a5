// RMS norm of queries and keys for each head, and the position's rotation, in one
// pass.  Per token and head x of D elements:
//   hat = x rstd, rstd = 1 / sqrt(mean(x^2) + eps),   n = hat w,
// then the R first elements turned in pairs (n1, n2) by the position's angles,
//   y1 = n1 cos - n2 sin,   y2 = n2 cos + n1 sin,
// pairs being elements i and i + R / 2, or 2 i and 2 i + 1 (interleaved).
// Backward: dn = dy turned back, dx = rstd (w dn - hat mean(w dn hat)),
// dw = sum over tokens and heads of dn hat.
#include "mgs_lm.h"
#include "mgs_num.cuh"

namespace mgs {
namespace {

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

struct Rows {
    const void *x, *w, *gy;
    void *out;        // forward: y; backward: dx
    int64_t xs[3], gs[3];
    int H;
};
struct Args {
    Rows r[2];        // queries, keys
    const float *table;
    const int32_t *positions;
    int64_t ps[2], rows, B, T;
    int D, R, interleaved;
    float eps;
};

// one warp a head, a lane's pairs 32 apart
template <typename T, bool BWD>
__global__ void __launch_bounds__(256) qk_norm_kernel(Args a, float *part) {
    const int lane = threadIdx.x & 31, half = a.R / 2, heads = a.r[0].H + a.r[1].H;
    const int64_t tokens = a.B * a.T, warps = int64_t(gridDim.x) * 8;
    float sums[2][4][2] = {};
    for (int64_t i = int64_t(blockIdx.x) * 8 + threadIdx.x / 32; i < tokens * heads; i += warps) {
        const int64_t tok = i / heads, b = tok / a.T, t = tok % a.T;
        const int hh = int(i % heads), which = hh >= a.r[0].H, h = which ? hh - a.r[0].H : hh;
        const Rows &r = a.r[which];
        const T *x = (const T *)r.x + b * r.xs[0] + t * r.xs[1] + h * r.xs[2], *w = (const T *)r.w;
        T *out = (T *)r.out + (tok * r.H + h) * a.D;
        const int64_t at = a.positions ? a.positions[b * a.ps[0] + t * a.ps[1]] : t;
        const bool live = a.R == 0 || (at >= 0 && at < a.rows);
        float v[4][2], sum = 0.f;
        for (int j = 0; j < 4; ++j) {
            const int p = lane + 32 * j;
            if (2 * p >= a.D) break;
            const int e1 = p < half ? (a.interleaved ? 2 * p : p) : 2 * p, e2 = p < half && !a.interleaved ? p + half : e1 + 1;
            v[j][0] = to_f(x[e1]), v[j][1] = to_f(x[e2]);
            sum = fmaf(v[j][0], v[j][0], fmaf(v[j][1], v[j][1], sum));
        }
        const float rstd = rsqrtf(warp_sum(sum) / float(a.D) + a.eps);
        float g[4][2], dot = 0.f;
        for (int j = 0; j < 4; ++j) {
            const int p = lane + 32 * j;
            if (2 * p >= a.D) break;
            const int e1 = p < half ? (a.interleaved ? 2 * p : p) : 2 * p, e2 = p < half && !a.interleaved ? p + half : e1 + 1;
            const float w1 = w ? to_f(w[e1]) : 1.f, w2 = w ? to_f(w[e2]) : 1.f;
            float c = 1.f, s = 0.f;
            if (p < half && live) c = a.table[at * a.R + p], s = a.table[at * a.R + half + p];
            v[j][0] *= rstd, v[j][1] *= rstd;
            if (!BWD) {
                const float n1 = v[j][0] * w1, n2 = v[j][1] * w2;
                out[e1] = from_f<T>(live ? n1 * c - n2 * s : 0.f);
                out[e2] = from_f<T>(live ? n2 * c + n1 * s : 0.f);
            } else {
                const T *gy = (const T *)r.gy + b * r.gs[0] + t * r.gs[1] + h * r.gs[2];
                const float g1 = live ? to_f(gy[e1]) : 0.f, g2 = live ? to_f(gy[e2]) : 0.f;
                const float d1 = g1 * c + g2 * s, d2 = g2 * c - g1 * s;
                if (live) sums[which][j][0] += d1 * v[j][0], sums[which][j][1] += d2 * v[j][1];
                g[j][0] = d1 * w1, g[j][1] = d2 * w2;
                dot += g[j][0] * v[j][0] + g[j][1] * v[j][1];
            }
        }
        if (BWD) {
            dot = warp_sum(dot) / float(a.D);
            for (int j = 0; j < 4; ++j) {
                const int p = lane + 32 * j;
                if (2 * p >= a.D) break;
                const int e1 = p < half ? (a.interleaved ? 2 * p : p) : 2 * p, e2 = p < half && !a.interleaved ? p + half : e1 + 1;
                out[e1] = from_f<T>(live ? rstd * (g[j][0] - v[j][0] * dot) : 0.f);
                out[e2] = from_f<T>(live ? rstd * (g[j][1] - v[j][1] * dot) : 0.f);
            }
        }
    }
    if (BWD) {
        for (int which = 0; which < 2; ++which)
            for (int j = 0; j < 4; ++j) {
                const int p = lane + 32 * j;
                if (2 * p >= a.D) break;
                const int e1 = p < half ? (a.interleaved ? 2 * p : p) : 2 * p, e2 = p < half && !a.interleaved ? p + half : e1 + 1;
                float *row = part + ((int64_t(blockIdx.x) * 8 + threadIdx.x / 32) * 2 + which) * a.D;
                row[e1] = sums[which][j][0], row[e2] = sums[which][j][1];
            }
    }
}

// dw[which][e] = the sum over `parts` rows, one warp a column
template <typename T>
__global__ void qk_dw_kernel(const float *part, T *dwq, T *dwk, int parts, int D) {
    const int col = blockIdx.x * 8 + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (col >= 2 * D) return;
    float s = 0.f;
    for (int i = lane; i < parts; i += 32) s += part[int64_t(i) * 2 * D + col];
    s = warp_sum(s);
    T *dw = col < D ? dwq : dwk;
    if (lane == 0 && dw) dw[col % D] = from_f<T>(s);
}

int64_t blocks_of(int64_t rows) { return min64((rows + 7) / 8, 152 * 8); }

Args args_of(const mgs_qk_norm_shape &sh, const void *q, const void *k, const void *qw, const void *kw,
             const void *gq, const void *gk, const float *table, const int32_t *positions, void *oq, void *ok) {
    Args a = {};
    a.r[0] = {q, qw, gq, oq, {}, {}, int(sh.Hq)}, a.r[1] = {k, kw, gk, ok, {}, {}, int(sh.Hk)};
    for (int i = 0; i < 3; ++i) {
        a.r[0].xs[i] = sh.q_stride[i], a.r[1].xs[i] = sh.k_stride[i];
        a.r[0].gs[i] = sh.gq_stride[i], a.r[1].gs[i] = sh.gk_stride[i];
    }
    a.table = table, a.positions = positions, a.ps[0] = sh.pos_stride[0], a.ps[1] = sh.pos_stride[1];
    a.rows = sh.positions, a.B = sh.B, a.T = sh.T, a.D = sh.D, a.R = sh.rotary, a.interleaved = sh.interleaved,
    a.eps = sh.eps;
    return a;
}

}  // namespace

cudaError_t launch_qk_norm_fwd(const mgs_qk_norm_shape &sh, const void *q, const void *k, const void *qw,
                               const void *kw, const float *table, const int32_t *positions, void *yq, void *yk,
                               cudaStream_t s) {
    const Args a = args_of(sh, q, k, qw, kw, nullptr, nullptr, table, positions, yq, yk);
    const unsigned grid = unsigned(blocks_of(sh.B * sh.T * (sh.Hq + sh.Hk)));
    if (sh.dtype == MGS_BF16) qk_norm_kernel<bf16, false><<<grid, 256, 0, s>>>(a, nullptr);
    else qk_norm_kernel<float, false><<<grid, 256, 0, s>>>(a, nullptr);
    return cudaGetLastError();
}

size_t qk_norm_bwd_workspace_bytes(const mgs_qk_norm_shape &sh) {
    return size_t(blocks_of(sh.B * sh.T * (sh.Hq + sh.Hk))) * 8 * 2 * size_t(sh.D) * 4;
}

cudaError_t launch_qk_norm_bwd(const mgs_qk_norm_shape &sh, const void *q, const void *k, const void *qw,
                               const void *kw, const void *gq, const void *gk, const float *table,
                               const int32_t *positions, void *dq, void *dk, void *dqw, void *dkw, void *ws,
                               cudaStream_t s) {
    const Args a = args_of(sh, q, k, qw, kw, gq, gk, table, positions, dq, dk);
    const unsigned grid = unsigned(blocks_of(sh.B * sh.T * (sh.Hq + sh.Hk)));
    float *part = static_cast<float *>(ws);
    if (sh.dtype == MGS_BF16) qk_norm_kernel<bf16, true><<<grid, 256, 0, s>>>(a, part);
    else qk_norm_kernel<float, true><<<grid, 256, 0, s>>>(a, part);
    if (dqw || dkw) {
        if (sh.dtype == MGS_BF16)
            qk_dw_kernel<bf16><<<(2 * sh.D + 7) / 8, 256, 0, s>>>(part, (bf16 *)dqw, (bf16 *)dkw, int(grid) * 8, sh.D);
        else
            qk_dw_kernel<float><<<(2 * sh.D + 7) / 8, 256, 0, s>>>(part, (float *)dqw, (float *)dkw, int(grid) * 8, sh.D);
    }
    return cudaGetLastError();
}

}  // namespace mgs
