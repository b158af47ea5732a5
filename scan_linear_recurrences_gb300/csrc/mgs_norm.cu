// RMS norm with the residual's addition.  Per row of N:
//   r = x + res (rounded to the type: the residual stream that the next layer adds to),
//   rstd = 1 / sqrt(mean(r^2) + eps),   y = r rstd w,
// or y in fp8 (e4m3) with a scale for each row or each 128 columns,
//   scale = max|y| / 448,   q = y / scale.
// Backward, with hat = r rstd:
//   dx = rstd (w dy - hat mean(w dy hat)) + dr,   dw = sum over rows of dy hat
// (dx is the gradient of x and of res alike).  All sums in fp32.  Bound by
// memory: each tensor is read or written once, a row stays in registers
// between the sum and its use.
#include "mgs_lm.h"
#include "mgs_num.cuh"

namespace mgs {
namespace {

constexpr float kFp8Max = 448.f;

// Sums (SUM) or maxima over the `TPR` threads of a row: TPR <= 32 within a
// warp, else the whole block.
template <bool SUM>
__device__ __forceinline__ float comb(float a, float b) { return SUM ? a + b : fmaxf(a, b); }
template <bool SUM>
__device__ __forceinline__ float row_reduce(float x, int tpr, float *red) {
    for (int m = min(tpr, 32) >> 1; m > 0; m >>= 1) x = comb<SUM>(x, __shfl_xor_sync(0xffffffffu, x, m));
    if (tpr <= 32) return x;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    float t = red[0];
    for (int i = 1; i < tpr / 32; ++i) t = comb<SUM>(t, red[i]);
    return t;
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t u;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(u) : "f"(hi), "f"(lo));
    return u;
}

// V consecutive elements as one access (16 bytes), or V = 1: any N, any alignment
template <typename T, int V>
__device__ __forceinline__ void get(const T *p, float (&v)[V]) {
    if constexpr (V == 1)
        v[0] = to_f(*p);
    else
        unpack(*reinterpret_cast<const uint4 *>(p), v);
}
template <typename T, int V>
__device__ __forceinline__ void put(T *p, const float (&v)[V]) {
    if constexpr (V == 1)
        *p = from_f<T>(v[0]);
    else
        *reinterpret_cast<uint4 *>(p) = pack(v);
}
template <int V>
__device__ __forceinline__ void put8(uint8_t *p, const float (&v)[V]) {
    if constexpr (V == 1) {
        *p = uint8_t(e4m3x2(v[0], 0.f));
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<uint32_t *>(p + i) = e4m3x2(v[i], v[i + 1]) | (e4m3x2(v[i + 2], v[i + 3]) << 16);
    }
}

// TPR threads a row, blockDim / TPR rows a block, NV pieces of V elements a
// thread.  FP8: 0 y in the type, 1 a scale a row, 2 a scale for 128 columns.
template <typename T, int V, int NV, int FP8>
__global__ void __launch_bounds__(1024)
    norm_fwd_kernel(const T *__restrict__ x, const T *__restrict__ res, const T *__restrict__ w, float eps,
                    T *__restrict__ ro, T *__restrict__ y, float *__restrict__ rstd_out, uint8_t *__restrict__ q8,
                    float *__restrict__ scales, int64_t rows, int N, int tpr) {
    __shared__ float red[2][32];
    const int c = threadIdx.x % tpr;
    const int64_t row = int64_t(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool live = row < rows;
    float r[NV][V], ww[NV][V], sum = 0.f, top = 0.f;
    const int64_t at = row * N;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (c + i * tpr) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) r[i][j] = ww[i][j] = 0.f;
        if (live && e < N) {
            get<T, V>(x + at + e, r[i]);
            get<T, V>(w + e, ww[i]);
            if (res) {
                float a[V];
                get<T, V>(res + at + e, a);
#pragma unroll
                for (int j = 0; j < V; ++j) r[i][j] = to_f(from_f<T>(r[i][j] + a[j]));
                put<T, V>(ro + at + e, r[i]);
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                sum = fmaf(r[i][j], r[i][j], sum);
                if (FP8 == 1) top = fmaxf(top, fabsf(r[i][j] * ww[i][j]));
            }
        }
    }
    sum = row_reduce<true>(sum, tpr, red[0]);
    const float rstd = rsqrtf(sum / float(N) + eps);
    if (FP8 == 0 && rstd_out && live && c == 0) rstd_out[row] = rstd;
    float inv = 0.f;
    if (FP8 == 1) {
        top = row_reduce<false>(top, tpr, red[1]) * rstd;
        const float sc = top * (1.f / kFp8Max);
        if (live && c == 0) scales[row] = sc;
        inv = sc > 0.f ? 1.f / sc : 1.f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (c + i * tpr) * V;
        const bool in = live && e < N;
#pragma unroll
        for (int j = 0; j < V; ++j) r[i][j] = r[i][j] * rstd * ww[i][j];
        if (FP8 == 0) {
            if (in) put<T, V>(y + at + e, r[i]);
            continue;
        }
        if (FP8 == 2) {
            // 128 / V neighbouring threads hold a group (V = 1 has its own kernel)
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < V; ++j) m = fmaxf(m, fabsf(r[i][j]));
#pragma unroll
            for (int s = 64 / V; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
            const float sc = m * (1.f / kFp8Max);
            if (in && e % 128 == 0) scales[row * (N / 128) + e / 128] = sc;
            inv = sc > 0.f ? 1.f / sc : 1.f;
        }
        if (in) {
#pragma unroll
            for (int j = 0; j < V; ++j) r[i][j] *= inv;
            put8<V>(q8 + at + e, r[i]);
        }
    }
}

// Any N and alignment, one block a row, the row read again for each use.
template <typename T, int FP8>
__global__ void __launch_bounds__(256)
    norm_fwd_any_kernel(const T *__restrict__ x, const T *__restrict__ res, const T *__restrict__ w, float eps, T *ro,
                        T *__restrict__ y, float *__restrict__ rstd_out, uint8_t *__restrict__ q8,
                        float *__restrict__ scales, int64_t rows, int64_t N) {
    __shared__ float red[2][32];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const int64_t at = row * N;
        const T *r = res ? ro : x;
        float sum = 0.f, top = 0.f;
        for (int64_t e = threadIdx.x; e < N; e += 256) {
            float a = to_f(x[at + e]);
            if (res) {
                const T t = from_f<T>(a + to_f(res[at + e]));
                ro[at + e] = t;
                a = to_f(t);
            }
            sum = fmaf(a, a, sum);
            if (FP8 == 1) top = fmaxf(top, fabsf(a * to_f(w[e])));
        }
        sum = row_reduce<true>(sum, 256, red[0]);
        const float rstd = rsqrtf(sum / float(N) + eps);
        if (FP8 == 0 && rstd_out && threadIdx.x == 0) rstd_out[row] = rstd;
        float inv = 0.f;
        if (FP8 == 1) {
            const float sc = row_reduce<false>(top, 256, red[1]) * rstd * (1.f / kFp8Max);
            if (threadIdx.x == 0) scales[row] = sc;
            inv = sc > 0.f ? 1.f / sc : 1.f;
        }
        if (FP8 == 2) {  // N is a multiple of 128: one warp a group
            for (int64_t g = threadIdx.x / 32; g < N / 128; g += 8) {
                float v[4], m = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t e = g * 128 + 32 * j + (threadIdx.x & 31);
                    // written by other threads of this block, before the barrier of the sum
                    v[j] = to_f(r[at + e]) * rstd * to_f(w[e]);
                    m = fmaxf(m, fabsf(v[j]));
                }
                for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
                const float sc = m * (1.f / kFp8Max), iv = sc > 0.f ? 1.f / sc : 1.f;
                if ((threadIdx.x & 31) == 0) scales[row * (N / 128) + g] = sc;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    q8[at + g * 128 + 32 * j + (threadIdx.x & 31)] = uint8_t(e4m3x2(v[j] * iv, 0.f));
            }
        } else {
            for (int64_t e = threadIdx.x; e < N; e += 256) {
                const float v = to_f(r[at + e]) * rstd * to_f(w[e]);
                if (FP8 == 0)
                    y[at + e] = from_f<T>(v);
                else
                    q8[at + e] = uint8_t(e4m3x2(v * inv, 0.f));
            }
        }
        __syncthreads();
    }
}

// A block walks rows blockIdx, + gridDim, ..; dw's sums over its rows stay in
// registers and go to part[block][N] at the end.
template <typename T, int V, int NV>
__global__ void __launch_bounds__(1024)
    norm_bwd_kernel(const T *__restrict__ r, const T *__restrict__ w, const float *__restrict__ rstd,
                    const T *__restrict__ gy, const T *__restrict__ gr, T *__restrict__ dx, float *__restrict__ part,
                    int64_t rows, int N) {
    __shared__ float red[2][32];
    const int tpr = blockDim.x, c = threadIdx.x;
    float dw[NV][V], ww[NV][V];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (c + i * tpr) * V;
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = ww[i][j] = 0.f;
        if (e < N) get<T, V>(w + e, ww[i]);
    }
    int turn = 0;  // two reduction buffers: one barrier a row
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x, turn ^= 1) {
        const int64_t at = row * N;
        const float rs = rstd[row];
        float hat[NV][V], g[NV][V], dot = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (c + i * tpr) * V;
            if (e < N) {
                get<T, V>(r + at + e, hat[i]);
                get<T, V>(gy + at + e, g[i]);
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) hat[i][j] = g[i][j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < V; ++j) {
                hat[i][j] *= rs;
                dw[i][j] = fmaf(g[i][j], hat[i][j], dw[i][j]);
                g[i][j] *= ww[i][j];
                dot = fmaf(g[i][j], hat[i][j], dot);
            }
        }
        dot = row_reduce<true>(dot, tpr, red[turn]) / float(N);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (c + i * tpr) * V;
            if (e >= N) continue;
            float o[V], a[V];
            if (gr) get<T, V>(gr + at + e, a);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                o[j] = rs * (g[i][j] - hat[i][j] * dot);
                if (gr) o[j] += a[j];
            }
            put<T, V>(dx + at + e, o);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (c + i * tpr) * V;
        if (e < N)
#pragma unroll
            for (int j = 0; j < V; ++j) part[int64_t(blockIdx.x) * N + e + j] = dw[i][j];
    }
}

// Any N and alignment; dw's sums of a block in part[block][N] (its own row, zeroed here)
template <typename T>
__global__ void __launch_bounds__(256)
    norm_bwd_any_kernel(const T *__restrict__ r, const T *__restrict__ w, const float *__restrict__ rstd,
                        const T *__restrict__ gy, const T *__restrict__ gr, T *__restrict__ dx,
                        float *__restrict__ part, int64_t rows, int64_t N) {
    __shared__ float red[32];
    float *dw = part + int64_t(blockIdx.x) * N;
    for (int64_t e = threadIdx.x; e < N; e += 256) dw[e] = 0.f;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const int64_t at = row * N;
        const float rs = rstd[row];
        float dot = 0.f;
        for (int64_t e = threadIdx.x; e < N; e += 256)
            dot = fmaf(to_f(gy[at + e]) * to_f(w[e]), to_f(r[at + e]) * rs, dot);
        __syncthreads();
        dot = row_reduce<true>(dot, 256, red) / float(N);
        for (int64_t e = threadIdx.x; e < N; e += 256) {
            const float hat = to_f(r[at + e]) * rs, g = to_f(gy[at + e]);
            dw[e] = fmaf(g, hat, dw[e]);
            const float o = rs * (g * to_f(w[e]) - hat * dot);
            dx[at + e] = from_f<T>(gr ? o + to_f(gr[at + e]) : o);
        }
    }
}

// dw[n] = sum over blocks of part[block][n], in a fixed order: 32 columns and
// 8 runs of blocks a thread block
template <typename T>
__global__ void __launch_bounds__(256)
    norm_dw_kernel(const float *__restrict__ part, T *__restrict__ dw, int blocks, int64_t N) {
    __shared__ float red[8][33];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t n = int64_t(blockIdx.x) * 32 + c;
    float s = 0.f;
    if (n < N)
        for (int i = k; i < blocks; i += 8) s += part[int64_t(i) * N + n];
    red[k][c] = s;
    __syncthreads();
    if (k == 0 && n < N) {
        for (int i = 1; i < 8; ++i) s += red[i][c];
        dw[n] = from_f<T>(s);
    }
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Threads a row and pieces a thread: up to 4 pieces, at least a warp.
struct Shape {
    int tpr, nv;
};
Shape shape_of(int64_t pieces) {
    Shape s{32, 1};
    while (int64_t(s.tpr) * s.nv < pieces) {
        if (s.tpr < 256)
            s.tpr *= 2;
        else if (s.nv < 4)
            s.nv *= 2;
        else if (s.tpr < 1024)
            s.tpr *= 2;
        else
            return {0, 0};
    }
    return s;
}

template <typename T, int FP8>
cudaError_t fwd_go(const T *x, const T *res, const T *w, float eps, T *r, T *y, float *rstd, uint8_t *q8,
                   float *scales, int64_t rows, int64_t N, cudaStream_t s) {
    constexpr int V = kVec<T>;
    const Shape sh = shape_of((N + V - 1) / V);
    const bool vec = N % V == 0 && al16(x) && al16(res) && al16(w) && al16(r) && al16(y) && al16(q8) && sh.tpr > 0;
    if (!vec) {
        const unsigned grid = unsigned(min64(rows, 152 * 8));
        norm_fwd_any_kernel<T, FP8><<<grid, 256, 0, s>>>(x, res, w, eps, r, y, rstd, q8, scales, rows, N);
        return cudaGetLastError();
    }
    const int rpb = sh.tpr > 32 ? 1 : 4;  // rows of a block: a row's threads are one warp, or the whole block
    const int64_t grid = (rows + rpb - 1) / rpb;
    if (grid > 0x7fffffff) return cudaErrorInvalidConfiguration;
#define MGS_GO(NV)                                                                                              \
    norm_fwd_kernel<T, V, NV, FP8><<<unsigned(grid), unsigned(rpb * sh.tpr), 0, s>>>(x, res, w, eps, r, y, rstd, \
                                                                                    q8, scales, rows, int(N), sh.tpr)
    if (sh.nv == 1) MGS_GO(1);
    else if (sh.nv == 2) MGS_GO(2);
    else MGS_GO(4);
#undef MGS_GO
    return cudaGetLastError();
}

int bwd_blocks(int64_t rows) { return int(min64(rows, 152 * 4)); }

template <typename T>
cudaError_t bwd_go(const T *r, const T *w, const float *rstd, const T *gy, const T *gr, T *dx, T *dw, int64_t rows,
                   int64_t N, float *part, cudaStream_t s) {
    constexpr int V = kVec<T>;
    const Shape sh = shape_of((N + V - 1) / V);
    const bool vec = N % V == 0 && al16(r) && al16(w) && al16(gy) && al16(gr) && al16(dx) && sh.tpr > 0;
    const int blocks = bwd_blocks(rows);
    if (!vec)
        norm_bwd_any_kernel<T><<<blocks, 256, 0, s>>>(r, w, rstd, gy, gr, dx, part, rows, N);
    else if (sh.nv == 1)
        norm_bwd_kernel<T, V, 1><<<blocks, sh.tpr, 0, s>>>(r, w, rstd, gy, gr, dx, part, rows, int(N));
    else if (sh.nv == 2)
        norm_bwd_kernel<T, V, 2><<<blocks, sh.tpr, 0, s>>>(r, w, rstd, gy, gr, dx, part, rows, int(N));
    else
        norm_bwd_kernel<T, V, 4><<<blocks, sh.tpr, 0, s>>>(r, w, rstd, gy, gr, dx, part, rows, int(N));
    norm_dw_kernel<T><<<unsigned((N + 31) / 32), 256, 0, s>>>(part, dw, blocks, N);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rms_norm_fwd(int dtype, const void *x, const void *res, const void *w, float eps, void *r, void *y,
                                float *rstd, int64_t rows, int64_t N, cudaStream_t s) {
    if (dtype == MGS_BF16)
        return fwd_go<bf16, 0>((const bf16 *)x, (const bf16 *)res, (const bf16 *)w, eps, (bf16 *)r, (bf16 *)y, rstd,
                               nullptr, nullptr, rows, N, s);
    return fwd_go<float, 0>((const float *)x, (const float *)res, (const float *)w, eps, (float *)r, (float *)y, rstd,
                            nullptr, nullptr, rows, N, s);
}

template <typename T>
static cudaError_t fp8_go(const void *x, const void *res, const void *w, float eps, void *r, void *q8, float *scales,
                          int64_t rows, int64_t N, int group, cudaStream_t s) {
    if (group)
        return fwd_go<T, 2>((const T *)x, (const T *)res, (const T *)w, eps, (T *)r, nullptr, nullptr, (uint8_t *)q8,
                            scales, rows, N, s);
    return fwd_go<T, 1>((const T *)x, (const T *)res, (const T *)w, eps, (T *)r, nullptr, nullptr, (uint8_t *)q8,
                        scales, rows, N, s);
}

cudaError_t launch_rms_norm_fp8(int dtype, const void *x, const void *res, const void *w, float eps, void *r,
                                void *q8, float *scales, int64_t rows, int64_t N, int group, cudaStream_t s) {
    return dtype == MGS_BF16 ? fp8_go<bf16>(x, res, w, eps, r, q8, scales, rows, N, group, s)
                             : fp8_go<float>(x, res, w, eps, r, q8, scales, rows, N, group, s);
}

size_t rms_norm_bwd_workspace_bytes(int64_t rows, int64_t N) { return size_t(bwd_blocks(rows)) * size_t(N) * 4; }

cudaError_t launch_rms_norm_bwd(int dtype, const void *r, const void *w, const float *rstd, const void *gy,
                                const void *gr, void *dx, void *dw, int64_t rows, int64_t N, void *ws,
                                cudaStream_t s) {
    float *part = static_cast<float *>(ws);
    if (dtype == MGS_BF16)
        return bwd_go<bf16>((const bf16 *)r, (const bf16 *)w, rstd, (const bf16 *)gy, (const bf16 *)gr, (bf16 *)dx,
                            (bf16 *)dw, rows, N, part, s);
    return bwd_go<float>((const float *)r, (const float *)w, rstd, (const float *)gy, (const float *)gr, (float *)dx,
                         (float *)dw, rows, N, part, s);
}

}  // namespace mgs
