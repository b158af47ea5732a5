// RMS norm with the residual's addition.  Per row of N:
//   r = x + res (rounded to the type: the residual stream that the next layer adds to),
//   rstd = 1 / sqrt(mean(r^2) + eps),   y = r rstd w,
// or y in fp8 (e4m3) with a scale for each row or each 128 columns,
//   scale = max|y| / 448,   q = y / scale.
// Backward, with hat = r rstd:
//   dx = rstd (w dy - hat mean(w dy hat)) + dr,   dw = sum over rows of dy hat
// (dx is the gradient of x and of res alike).  All sums in fp32.  Bound by
// memory: each tensor is read or written once, a row stays in registers
// between the sum and its use.  32768 rows of 2048 in bf16: forward 87 us a call
// (537 MB, 6.2 TB/s), backward 91 (5.9 TB/s) with dw's last sums; 8191 rows of
// 5120 to fp8 48.5 us (294 MB, 6.1 TB/s; groups of 128 52); one row of 4096 2.6 us
// on the device.
#include <cstring>
#include <type_traits>

#include "mgs_lm.h"
#include "mgs_num.cuh"
#include "mgs_rows.h"

namespace mgs {
namespace {

constexpr float kFp8Max = 448.f;

// The larger of two, NaN if either is: a NaN among a row's or group's values has
// to reach its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// The sum (MAX: the maximum) over the `tpr` threads of a row: tpr <= 32 within a
// warp, else the whole block, in one barrier.
template <bool MAX = false>
__device__ __forceinline__ float row_reduce(float x, int tpr, float *red) {
    auto join = [](float a, float b) { return MAX ? max_nan(a, b) : a + b; };
    for (int m = min(tpr, 32) >> 1; m > 0; m >>= 1) x = join(x, __shfl_xor_sync(0xffffffffu, x, m));
    if (tpr <= 32) return x;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    x = red[0];
    for (int i = 1; i < tpr / 32; ++i) x = join(x, red[i]);
    return x;
}

// The scale of values whose largest is `top`, and their quotients by it (by 1
// where it is zero), as products with the reciprocal: that differs from the
// quotient's own rounding where e4m3's rounding is a tie, and is as near.  A low
// scale, whose reciprocal would be infinite, and what it divides are first
// multiplied by 2^64 (in a branch: another product for every element costs 2 us of 52).
struct Scale {
    float scale, inv;
    bool low;
    __device__ __forceinline__ explicit Scale(float top) : scale(top * (1.f / kFp8Max)) {
        low = scale > 0.f && scale < 0x1p-64f;
        inv = 1.f / (low ? scale * 0x1p64f : scale > 0.f ? scale : 1.f);
    }
    template <int V>
    __device__ __forceinline__ void divide(float (&v)[V]) const {
        if (__builtin_expect(low, 0)) {
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] *= 0x1p64f;
        }
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] *= inv;
    }
};

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t u;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(u) : "f"(hi), "f"(lo));
    return u;
}

// 16 bytes that are read once (past L1), and written once
__device__ __forceinline__ uint4 load_once(const void *p) {
    uint4 u;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    return u;
}
__device__ __forceinline__ void store_once(void *p, const uint4 &u) { __stcs(reinterpret_cast<uint4 *>(p), u); }

template <int V>
__device__ __forceinline__ void put8(uint8_t *p, const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
        *reinterpret_cast<uint32_t *>(p + i) = e4m3x2(v[i], v[i + 1]) | (e4m3x2(v[i + 2], v[i + 3]) << 16);
}

// The V elements from column e of a row, as one piece of 16 bytes.  SHIFT: N is no
// multiple of V, so that rows start anywhere; a row's pieces are then those of
// the whole tensor that it lies in, the first one starting `s` elements before
// the row, and what of them is the neighbouring rows' is masked.  s is the same
// for all of a thread's rows: they are a multiple of V rows apart.
// (32768 rows of 1001 in bf16, element by element: forward 118 us, backward 208;
// so: 51 and 61.)
template <typename T, bool SHIFT>
struct Window {
    static constexpr int V = kVec<T>;
    const int64_t rows;
    const int N, s;
    __device__ __forceinline__ Window(int64_t row, int64_t rows_, int N_)
        : rows(rows_), N(N_), s(SHIFT ? int((row * N_) % V) : 0) {}
    // the piece's elements lo .. hi - 1 are the row's
    __device__ __forceinline__ int lo(int e) const { return max(0, s - e); }
    __device__ __forceinline__ int hi(int e) const { return min(V, N + s - e); }
    __device__ __forceinline__ uint4 load(const T *p, int64_t row, int e) const {
        if (row >= rows || e >= N + s) return make_uint4(0u, 0u, 0u, 0u);
        const T *at = p + row * N + (e - s);
        if (!SHIFT || (rows - row) * N - (e - s) >= V) return load_once(at);
        T v[V];  // the tensor ends within the piece
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = j < hi(e) ? at[j] : from_f<T>(0.f);
        uint4 u;
        memcpy(&u, v, 16);
        return u;
    }
    __device__ __forceinline__ void mask(int e, float (&v)[V]) const {
        if (!SHIFT) return;
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = j >= lo(e) && j < hi(e) ? v[j] : 0.f;
    }
    __device__ __forceinline__ uint4 weight(const T *w, int e) const {
        if (!SHIFT) return e < N ? *reinterpret_cast<const uint4 *>(w + e) : make_uint4(0u, 0u, 0u, 0u);
        T v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = j >= lo(e) && j < hi(e) ? w[e - s + j] : from_f<T>(0.f);
        uint4 u;
        memcpy(&u, v, 16);
        return u;
    }
    __device__ __forceinline__ void store(T *p, int64_t row, int e, const uint4 &u) const {
        if (row >= rows || e >= N + s) return;
        T *at = p + row * N + (e - s);
        if (!SHIFT || (e >= s && N + s - e >= V)) {
            store_once(at, u);
            return;
        }
        T v[V];
        memcpy(v, &u, 16);
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j >= lo(e) && j < hi(e)) at[j] = v[j];
    }
    __device__ __forceinline__ void store8(uint8_t *p, int64_t row, int e, const float (&v)[V]) const {
        if (row >= rows || e >= N + s) return;
        uint8_t *at = p + row * N + (e - s);
        if (!SHIFT || (e >= s && N + s - e >= V)) {
            put8<V>(at, v);
            return;
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j >= lo(e) && j < hi(e)) at[j] = uint8_t(e4m3x2(v[j], 0.f));
    }
    // fp32 sums of the row's columns, into a row of N of them
    __device__ __forceinline__ void store_sums(float *p, int e, const float (&v)[V]) const {
        if (e >= N + s) return;
        if (!SHIFT) {
#pragma unroll
            for (int j = 0; j < V; j += 4)
                *reinterpret_cast<float4 *>(p + e + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
            return;
        }
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (j >= lo(e) && j < hi(e)) p[e - s + j] = v[j];
    }
};

// TPR threads a row, blockDim / TPR rows a block at a time, NV pieces of V
// elements (16 bytes) a thread.  A block walks rows, gridDim steps apart, and
// has the next row's loads in flight while it reduces and writes the current
// one's, w in registers (not with 8 pieces: they would not fit).  FP8: 0 y in the
// type, 1 a scale a row, 2 a scale for 128 columns.  SHIFT: rows of any length
// (Window).
template <typename T, int NV, int FP8, bool SHIFT>
__global__ void __launch_bounds__(NV == 1 ? 256 : 512, NV == 1 ? 4 : NV == 2 ? 2 : 1)
    norm_fwd_kernel(const T *__restrict__ x, const T *__restrict__ res, const T *__restrict__ w, float eps,
                    T *__restrict__ ro, T *__restrict__ y, float *__restrict__ rstd_out, uint8_t *__restrict__ q8,
                    float *__restrict__ scales, int64_t rows, int N, int tpr) {
    constexpr int V = kVec<T>;
    __shared__ float red[2][2][32];  // in turn: one barrier for a reduction (the sum's and the maximum's apart)
    const int c = threadIdx.x % tpr;
    RowWalk at(blockIdx.x, gridDim.x, threadIdx.x, blockDim.x, tpr);
    const float inv_n = 1.f / float(N);
    const Window<T, SHIFT> win(at.row, rows, N);
    uint4 ux[NV], ur[NV], uw[NV];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            ux[i] = win.load(x, row, (c + i * tpr) * V);
            if (res) ur[i] = win.load(res, row, (c + i * tpr) * V);
        }
    };
    fetch(at.row);
    constexpr bool PREFETCH = NV < 8;
    auto weight = [&](int i) { return win.weight(w, (c + i * tpr) * V); };
    if (PREFETCH) {
#pragma unroll
        for (int i = 0; i < NV; ++i) uw[i] = weight(i);
    }
    int turn = 0;
    for (; at.more(rows); at.next(), turn ^= 1) {
        const int64_t row = at.row;
        const bool live = row < rows;
        float r[NV][V], sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (c + i * tpr) * V;
            unpack(ux[i], r[i]);
            if (res) {
                float a[V];
                unpack(ur[i], a);
#pragma unroll
                for (int j = 0; j < V; ++j) r[i][j] += a[j];
                const uint4 u = pack(r[i]);
                win.store(ro, row, e, u);
                unpack(u, r[i]);
            }
            win.mask(e, r[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) sum = fmaf(r[i][j], r[i][j], sum);
        }
        if (PREFETCH) fetch(row + at.step);
        sum = row_reduce(sum, tpr, red[turn][0]);
        const float rstd = rsqrtf(sum * inv_n + eps);
        if (FP8 == 0 && rstd_out && live && c == 0) rstd_out[row] = rstd;
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (c + i * tpr) * V;
            float ww[V];
            unpack(PREFETCH ? uw[i] : weight(i), ww);
#pragma unroll
            for (int j = 0; j < V; ++j) r[i][j] = r[i][j] * rstd * ww[j];
            if (FP8 == 0) win.store(y, row, e, pack(r[i]));
            if (FP8 == 1) {
#pragma unroll
                for (int j = 0; j < V; ++j) top = max_nan(top, fabsf(r[i][j]));
            }
            if (FP8 == 2) {
                // 128 / V neighbouring threads hold a group
                float m = 0.f;
#pragma unroll
                for (int j = 0; j < V; ++j) m = max_nan(m, fabsf(r[i][j]));
#pragma unroll
                for (int s = 64 / V; s > 0; s >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, s));
                const Scale sc(m);
                if (live && e < N && e % 128 == 0) scales[row * (N / 128) + e / 128] = sc.scale;
                sc.divide(r[i]);
                win.store8(q8, row, e, r[i]);
            }
        }
        if (FP8 == 1) {
            const Scale sc(row_reduce<true>(top, tpr, red[turn][1]));
            if (live && c == 0) scales[row] = sc.scale;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                sc.divide(r[i]);
                win.store8(q8, row, (c + i * tpr) * V, r[i]);
            }
        }
        if (!PREFETCH) fetch(row + at.step);
    }
}

// Any N and alignment (tensors that do not start at a multiple of 16 bytes, rows too
// long for the registers), one block a row, the row read again for each use.
template <typename T, int FP8>
__global__ void __launch_bounds__(256)
    norm_fwd_any_kernel(const T *__restrict__ x, const T *__restrict__ res, const T *__restrict__ w, float eps, T *ro,
                        T *__restrict__ y, float *__restrict__ rstd_out, uint8_t *__restrict__ q8,
                        float *__restrict__ scales, int64_t rows, int64_t N) {
    __shared__ float red[2][32];
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const int64_t at = row * N;
        const T *r = res ? ro : x;
        float sum = 0.f;
        for (int64_t e = threadIdx.x; e < N; e += 256) {
            float a = to_f(x[at + e]);
            if (res) {
                const T t = from_f<T>(a + to_f(res[at + e]));
                ro[at + e] = t;
                a = to_f(t);
            }
            sum = fmaf(a, a, sum);
        }
        const float rstd = rsqrtf(row_reduce(sum, 256, red[0]) / float(N) + eps);
        if (FP8 == 0 && rstd_out && threadIdx.x == 0) rstd_out[row] = rstd;
        Scale sc(0.f);
        if (FP8 == 1) {
            float top = 0.f;  // (a thread's elements are the ones that it has written)
            for (int64_t e = threadIdx.x; e < N; e += 256) top = max_nan(top, fabsf(to_f(r[at + e]) * rstd * to_f(w[e])));
            sc = Scale(row_reduce<true>(top, 256, red[1]));
            if (threadIdx.x == 0) scales[row] = sc.scale;
        }
        if (FP8 == 2) {  // N is a multiple of 128: one warp a group
            for (int64_t g = threadIdx.x / 32; g < N / 128; g += 8) {
                float v[4], m = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t e = g * 128 + 32 * j + (threadIdx.x & 31);
                    // written by other threads of this block, before the barrier of the sum
                    v[j] = to_f(r[at + e]) * rstd * to_f(w[e]);
                    m = max_nan(m, fabsf(v[j]));
                }
                for (int s = 16; s > 0; s >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, s));
                const Scale of(m);
                if ((threadIdx.x & 31) == 0) scales[row * (N / 128) + g] = of.scale;
                of.divide(v);
#pragma unroll
                for (int j = 0; j < 4; ++j) q8[at + g * 128 + 32 * j + (threadIdx.x & 31)] = uint8_t(e4m3x2(v[j], 0.f));
            }
        } else {
            for (int64_t e = threadIdx.x; e < N; e += 256) {
                float v[1] = {to_f(r[at + e]) * rstd * to_f(w[e])};
                if (FP8 == 0) {
                    y[at + e] = from_f<T>(v[0]);
                } else {
                    sc.divide(v);
                    q8[at + e] = uint8_t(e4m3x2(v[0], 0.f));
                }
            }
        }
        __syncthreads();
    }
}

// A block walks rows, the next row's loads in flight while it works on the
// current one (PREFETCH; long rows of bf16 have no registers for it: 8192 rows
// of 8192 142 us, 3.8 TB/s, where 16384 of 4096 take 93).
// A row stays in registers as it was loaded and is unpacked twice.  dw's sums
// over a thread's rows stay in registers and go to part[..][N] at the end: a
// row of it for each row that the grid has in hand at a time.
template <typename T, int NV, bool SHIFT>
__global__ void __launch_bounds__(NV == 1 ? 256 : 512, NV == 1 ? 3 : 1)
    norm_bwd_kernel(const T *__restrict__ r, const T *__restrict__ w, const float *__restrict__ rstd,
                    const T *__restrict__ gy, const T *__restrict__ gr, T *__restrict__ dx, float *__restrict__ part,
                    int64_t rows, int N, int tpr) {
    constexpr int V = kVec<T>;
    constexpr bool PREFETCH = NV * V <= 16;
    __shared__ float red[2][32];
    const int c = threadIdx.x % tpr;
    griddep_launch();
    RowWalk at(blockIdx.x, gridDim.x, threadIdx.x, blockDim.x, tpr);
    const int64_t first = at.row;
    const float inv_n = 1.f / float(N);
    const Window<T, SHIFT> win(first, rows, N);
    float dw[NV][V], rs_next;
    uint4 uw[NV], ur[NV], ug[NV], ua[NV];
    auto fetch = [&](int64_t row) {
        rs_next = row < rows ? rstd[row] : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (c + i * tpr) * V;
            ur[i] = win.load(r, row, e);
            ug[i] = win.load(gy, row, e);
            if (gr && PREFETCH) ua[i] = win.load(gr, row, e);
        }
    };
    fetch(first);
    auto weight = [&](int i) { return win.weight(w, (c + i * tpr) * V); };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (PREFETCH) uw[i] = weight(i);
#pragma unroll
        for (int j = 0; j < V; ++j) dw[i][j] = 0.f;
    }
    int turn = 0;  // two reduction buffers: one barrier a row
    for (; at.more(rows); at.next(), turn ^= 1) {
        const int64_t row = at.row;
        const float rs = rs_next;
        float dot = 0.f;
        uint4 cr[NV], cg[NV], ca[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            cr[i] = ur[i], cg[i] = ug[i], ca[i] = ua[i];
            float hat[V], g[V], ww[V];
            unpack(cr[i], hat);
            unpack(cg[i], g);
            win.mask((c + i * tpr) * V, hat), win.mask((c + i * tpr) * V, g);
            unpack(PREFETCH ? uw[i] : weight(i), ww);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                hat[j] *= rs;
                dw[i][j] = fmaf(g[j], hat[j], dw[i][j]);
                dot = fmaf(g[j] * ww[j], hat[j], dot);
            }
        }
        if (PREFETCH) fetch(row + at.step);
        dot = row_reduce(dot, tpr, red[turn]) * inv_n;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (c + i * tpr) * V;
            float hat[V], g[V], ww[V], a[V];
            unpack(cr[i], hat);
            unpack(cg[i], g);
            unpack(PREFETCH ? uw[i] : weight(i), ww);
            if (gr) unpack(PREFETCH ? ca[i] : win.load(gr, row, e), a);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                g[j] = rs * (g[j] * ww[j] - hat[j] * rs * dot);
                if (gr) g[j] += a[j];
            }
            win.store(dx, row, e, pack(g));
        }
        if (!PREFETCH) fetch(row + at.step);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        win.store_sums(part + first * N, (c + i * tpr) * V, dw[i]);
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
        dot = row_reduce(dot, 256, red) / float(N);
        for (int64_t e = threadIdx.x; e < N; e += 256) {
            const float hat = to_f(r[at + e]) * rs, g = to_f(gy[at + e]);
            dw[e] = fmaf(g, hat, dw[e]);
            const float o = rs * (g * to_f(w[e]) - hat * dot);
            dx[at + e] = from_f<T>(gr ? o + to_f(gr[at + e]) : o);
        }
    }
}

// dw[n] = sum over blocks of part[block][n], in a fixed order: 32 columns and
// 32 runs of blocks a thread block
template <typename T>
__global__ void __launch_bounds__(1024)
    norm_dw_kernel(const float *__restrict__ part, T *__restrict__ dw, int blocks, int64_t N) {
    __shared__ float red[32][33];
    const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
    const int64_t n = int64_t(blockIdx.x) * 32 + c;
    griddep_wait();
    float s = 0.f;
    if (n < N) {
#pragma unroll 8
        for (int i = k; i < blocks; i += 32) s += part[int64_t(i) * N + n];
    }
    red[k][c] = s;
    __syncthreads();
    // warp k adds up column k
    s = red[c][k];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    const int64_t o = int64_t(blockIdx.x) * 32 + k;
    if (c == 0 && o < N) dw[o] = from_f<T>(s);
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Threads a row and pieces a thread.  Up to 32 pieces: a power of two of threads,
// several rows a warp.  Longer: whole warps.
struct Shape {
    int tpr, nv;
};
int64_t warps_of(int64_t pieces, int nv) { return (pieces + 32 * nv - 1) / (32 * nv); }
Shape shape_of(int64_t pieces, int nv) {
    if (pieces > 32) return {warps_of(pieces, nv) <= 16 ? int(32 * warps_of(pieces, nv)) : 0, nv};
    int t = 8;
    while (t < pieces) t *= 2;
    return {t, 1};
}
// Forward: four pieces a thread past 64, so that fewer warps wait for one another
// at a row's sum and a warp has more loads in flight (8191 rows of 5120 in bf16 to
// fp8: 160 threads of 4 48 us, 320 of 2 60; 30000 of 1024, a warp a row, 35,
// against 42 with 128 threads; 60000 of 512 44, a warp of 2 45); two where a
// quarter or more of four would lie idle (30000 of 768 in fp32 48 us, else 50).
Shape fwd_shape(int64_t pieces) {
    const int64_t w4 = warps_of(pieces, 4), w2 = warps_of(pieces, 2);
    return shape_of(pieces, pieces <= 64 ? 1 : pieces > 2048 ? 8 : 96 * w4 >= pieces && 2 * w4 > w2 ? 2 : 4);
}
// Backward: as many pieces as there are registers for with the next row's loads in
// flight (32768 rows of 2048 in bf16: 128 threads of 2 91 us, 256 of 1 98)
Shape bwd_shape(int64_t pieces) {
    return shape_of(pieces, pieces <= 192 ? 1 : pieces <= 640 ? 2 : pieces <= 2048 ? 4 : 8);
}
template <int N>
using Int = std::integral_constant<int, N>;
// Rows of a block: a row's threads are within a warp, or the whole block.
int block_rows(int tpr) { return tpr > 32 ? 1 : 128 / tpr; }

// Blocks an SM, of kernels that leave room for `most` threads there.  Where a
// thread has more than one row, the blocks are a multiple of 8 (as 152 is), and
// with them the rows between two of a thread's: a multiple of a piece's elements.
int64_t grid_of(int64_t rows, int rpb, int threads, int most) {
    return min64((rows + rpb - 1) / rpb, 152 * (threads >= most ? 1 : most / threads));
}

template <typename T, int FP8>
cudaError_t fwd_go(const T *x, const T *res, const T *w, float eps, T *r, T *y, float *rstd, uint8_t *q8,
                   float *scales, int64_t rows, int64_t N, cudaStream_t s) {
    constexpr int V = kVec<T>;
    const bool shift = N % V != 0;  // a row may then begin and end within a piece
    const Shape sh = fwd_shape(shift ? (N + 2 * V - 2) / V : N / V);
    const bool vec = al16(x) && al16(res) && al16(w) && al16(r) && al16(y) && al16(q8) && sh.tpr > 0;
    if (!vec) {
        const unsigned grid = unsigned(min64(rows, 152 * 8));
        norm_fwd_any_kernel<T, FP8><<<grid, 256, 0, s>>>(x, res, w, eps, r, y, rstd, q8, scales, rows, N);
        return cudaGetLastError();
    }
    const int rpb = block_rows(sh.tpr);
    const int64_t grid = grid_of(rows, rpb, rpb * sh.tpr, sh.nv <= 2 ? 1024 : 512);
    auto go = [&](auto nv) {
        auto *fn = norm_fwd_kernel<T, nv.value, FP8, false>;
        if constexpr (FP8 != 2)  // whose rows are whole groups
            if (shift) fn = norm_fwd_kernel<T, nv.value, FP8, true>;
        fn<<<unsigned(grid), unsigned(rpb * sh.tpr), 0, s>>>(x, res, w, eps, r, y, rstd, q8, scales, rows, int(N),
                                                             sh.tpr);
    };
    if (sh.nv == 1) go(Int<1>());
    else if (sh.nv == 2) go(Int<2>());
    else if (sh.nv == 4) go(Int<4>());
    else go(Int<8>());
    return cudaGetLastError();
}

// The backward's grid: blocks, of how many rows.  Each row in hand has a row of
// the workspace for its sums of dw.
// Short rows' blocks are small, and so are their sums: more of them (60000 rows of
// 512 in bf16: 49 us with 12 blocks an SM, 82 with 4).
int64_t bwd_blocks(int64_t N) {
    const int64_t n = N > 0 ? 6144 / N : 12;
    return 152 * (n < 4 ? 4 : n > 12 ? 12 : n);
}
int64_t bwd_parts(int64_t rows, int64_t N) { return min64(rows + 15, bwd_blocks(N) * (N <= 256 ? 16 : 1)); }

template <typename T>
cudaError_t bwd_go(const T *r, const T *w, const float *rstd, const T *gy, const T *gr, T *dx, T *dw, int64_t rows,
                   int64_t N, float *part, cudaStream_t s) {
    constexpr int V = kVec<T>;
    const bool shift = N % V != 0;
    const Shape sh = bwd_shape(shift ? (N + 2 * V - 2) / V : N / V);
    const bool vec = al16(r) && al16(w) && al16(gy) && al16(gr) && al16(dx) && al16(part) &&
                     sh.tpr > 0 && sh.nv < 8;
    int parts;
    if (!vec) {
        parts = int(min64(rows, bwd_blocks(N)));
        norm_bwd_any_kernel<T><<<parts, 256, 0, s>>>(r, w, rstd, gy, gr, dx, part, rows, N);
    } else {
        const int rpb = block_rows(sh.tpr), threads = rpb * sh.tpr;
        const int blocks =
            int(min64(bwd_blocks(N), grid_of(rows, rpb, threads, sh.nv == 1 ? 768 : 512)));
        parts = blocks * rpb;
        auto go = [&](auto nv) {
            auto *fn = shift ? norm_bwd_kernel<T, nv.value, true> : norm_bwd_kernel<T, nv.value, false>;
            fn<<<blocks, threads, 0, s>>>(r, w, rstd, gy, gr, dx, part, rows, int(N), sh.tpr);
        };
        if (sh.nv == 1) go(Int<1>());
        else if (sh.nv == 2) go(Int<2>());
        else go(Int<4>());
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_next(norm_dw_kernel<T>, unsigned((N + 31) / 32), 1024, 0, s, true, part, dw, parts, N);
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

size_t rms_norm_bwd_workspace_bytes(int64_t rows, int64_t N) { return size_t(bwd_parts(rows, N)) * size_t(N) * 4; }

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
