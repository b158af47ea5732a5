// RMS norm of queries and keys for each head, and the position's rotation, in one
// pass.  Per token and head x of D elements:
//   hat = x rstd, rstd = 1 / sqrt(mean(x^2) + eps),   n = hat w,
// then the R first elements turned in pairs (n1, n2) by the position's angles,
//   y1 = n1 cos - n2 sin,   y2 = n2 cos + n1 sin,
// pairs being elements i and i + R / 2, or 2 i and 2 i + 1 (interleaved).
// Backward: dn = dy turned back, dx = rstd (w dn - hat mean(w dn hat)),
// dw = sum over tokens and heads of dn hat.  Bound by memory: 8 x 4096 tokens of 16 + 16
// heads of 128 in bf16 85 us forward (6.3 TB/s), 123 backward (6.5).
//
// A lane holds both members of its pairs: two pieces of four elements of a head, four
// pairs, so that nothing but the sums passes between lanes.  G lanes (a power of two)
// share a head; a warp takes some of one token's queries, or keys, at a time, while the
// next ones and their row of the table are on their way to its part of shared memory;
// weights stay in its registers, and dw's sums over all that it sees.
#include <type_traits>

#include "mgs_launch.h"
#include "mgs_lm.h"
#include "mgs_num.cuh"

namespace mgs {
namespace {

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
    int64_t ps[2], rows, tokens, T;
    int D, R;
    int first;        // blocks from this one on work on the keys
    float eps;
};

// A warp's units of work: a token's heads in batches, one unit each.  From unit to unit
// by the step's own batches, tokens and sequences (no divisions on the way).
struct Walk {
    int b, t, batch, sb, st, sbatch, left;  // left: units from this one on, in steps of the grid
    __device__ __forceinline__ Walk(int64_t unit, int64_t step, int64_t tokens, int T, int batches) {
        const int64_t units = tokens * batches;
        left = unit < units ? int((units - unit + step - 1) / step) : 0;
        const int64_t tok = unit / batches, stok = step / batches;
        batch = int(unit - tok * batches), sbatch = int(step - stok * batches);
        b = int(tok / T), t = int(tok - int64_t(b) * T), sb = int(stok / T), st = int(stok - int64_t(sb) * T);
    }
    __device__ __forceinline__ void next(int T, int batches) {
        --left;
        batch += sbatch, t += st, b += sb;
        if (batch >= batches) batch -= batches, ++t;
        if (t >= T) t -= T, ++b;
    }
};

// Four elements of shared memory as two pairs of fp32 (zeros where `some` is not set), and back to memory
__device__ __forceinline__ void get4(const bf16 *p, bool some, f2 (&v)[2]) {
    uint2 u = *reinterpret_cast<const uint2 *>(p);
    if (!some) u = make_uint2(0u, 0u);
    v[0] = pair(bf_lo(u.x), bf_hi(u.x)), v[1] = pair(bf_lo(u.y), bf_hi(u.y));
}
__device__ __forceinline__ void get4(const float *p, bool some, f2 (&v)[2]) {
    float4 u = *reinterpret_cast<const float4 *>(p);
    if (!some) u = make_float4(0.f, 0.f, 0.f, 0.f);
    v[0] = pair(u.x, u.y), v[1] = pair(u.z, u.w);
}
template <bool VEC>
__device__ __forceinline__ void put4(bf16 *p, const f2 (&v)[2]) {
    const float2 a = both(v[0]), b = both(v[1]);
    const uint2 u = make_uint2(pack_bf16(a.x, a.y), pack_bf16(b.x, b.y));
    if (VEC) {
        __stcs(reinterpret_cast<uint2 *>(p), u);
    } else {
        uint16_t *q = reinterpret_cast<uint16_t *>(p);
        q[0] = uint16_t(u.x), q[1] = uint16_t(u.x >> 16), q[2] = uint16_t(u.y), q[3] = uint16_t(u.y >> 16);
    }
}
template <bool VEC>
__device__ __forceinline__ void put4(float *p, const f2 (&v)[2]) {
    const float2 a = both(v[0]), b = both(v[1]);
    if (VEC) __stcs(reinterpret_cast<float4 *>(p), make_float4(a.x, a.y, b.x, b.y));
    else p[0] = a.x, p[1] = a.y, p[2] = b.x, p[3] = b.y;
}

__device__ __forceinline__ void copy16(void *dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}

// One head's D elements to shared memory, by the G lanes of a head (VEC: whole pieces of 16 bytes, asynchronously)
template <typename T, int G, bool VEC>
__device__ __forceinline__ void copy_head(T *dst, const T *src, int D, int g) {
    if constexpr (VEC) {
        constexpr int V = kVec<T>;
#pragma unroll
        for (int i = 0; i < 8 / V; ++i)
            if ((g + i * G) * V < D) copy16(dst + (g + i * G) * V, src + (g + i * G) * V);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (g + i * G < D) dst[g + i * G] = src[g + i * G];
    }
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
    for (int m = G / 2; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    return x;
}

// The rotation of a lane's four pairs: members in a and b (elements i and i + R / 2), or
// neighbours (IL).  Backward by the opposite angle.
template <bool IL>
struct Turn;
template <>
struct Turn<false> {
    f2 c[2], s[2], ns[2];
    __device__ __forceinline__ void set(const float (&cos)[4], const float (&sin)[4]) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            c[i] = pair(cos[2 * i], cos[2 * i + 1]);
            s[i] = pair(sin[2 * i], sin[2 * i + 1]);
            ns[i] = pair(-sin[2 * i], -sin[2 * i + 1]);
        }
    }
    __device__ __forceinline__ void operator()(f2 (&a)[2], f2 (&b)[2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const f2 x = a[i], y = b[i];
            a[i] = fma2(y, ns[i], x * c[i]);
            b[i] = fma2(x, s[i], y * c[i]);
        }
    }
};
template <>
struct Turn<true> {
    f2 c[4], s[4];
    __device__ __forceinline__ void set(const float (&cos)[4], const float (&sin)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = pair(cos[i]), s[i] = pair(-sin[i], sin[i]);
    }
    __device__ __forceinline__ void operator()(f2 (&a)[2], f2 (&b)[2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float2 x = both(a[i]), y = both(b[i]);
            a[i] = fma2(pair(x.y, x.x), s[i], a[i] * c[i]);
            b[i] = fma2(pair(y.y, y.x), s[2 + i], b[i] * c[2 + i]);
        }
    }
};

// Heads that a lane works on in a unit, and units on their way at a time
template <typename T, bool BWD>
constexpr int kOnce = sizeof(T) == 2 ? 4 : BWD ? 1 : 2;
constexpr int kStages = 2;
// Bytes of a stage: 32 lanes of 8 elements, kOnce heads of one tensor or two, and a row of the table
template <typename T, bool BWD>
constexpr int kStageBytes = 256 * int(sizeof(T)) * kOnce<T, BWD> * (BWD ? 2 : 1) + 256 * 4;
// Blocks an SM (8 x 4096 tokens, 16 + 16 heads of 128 in bf16: forward 85 us with 2, 98 with
// 3; backward 123, and 141 with 3 of which two fit; fp32, 16 x 1000 tokens, 12 + 4 heads of
// 64: forward 23 and 20.6, backward 36 and 33).
template <typename T>
constexpr int kBlocksPerSm = sizeof(T) == 2 ? 2 : 3;

template <typename T, int G, bool VEC, bool IL, bool BWD>
__global__ void __launch_bounds__(256, kBlocksPerSm<T>)
    qk_norm_kernel(const __grid_constant__ Args a, float *__restrict__ part) {
    constexpr int P = 4, HEADS = 32 / G, U = kOnce<T, BWD>, HALF = 256 * U;  // HALF: elements of one tensor in a stage
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane % G, sub = lane / G;
    unsigned char *ring = smem + warp * (kStages * kStageBytes<T, BWD>);
    if (BWD) griddep_launch();
    const int k = int(blockIdx.x) >= a.first, block = int(blockIdx.x) - (k ? a.first : 0),
              blocks = k ? int(gridDim.x) - a.first : a.first;
    const Rows &r = a.r[k];
    const int half = a.R / 2, D = a.D, H = r.H, T_ = int(a.T);
    const bool in = 2 * P * g < D, turned = in && 2 * P * g < a.R;
    const int e1 = !turned || IL ? 2 * P * g : P * g, e2 = turned && !IL ? e1 + half : e1 + P;
    const float inv_d = 1.f / float(D);
    f2 w1[2], w2[2], dw1[2], dw2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const T *wk = (const T *)r.w;
        const bool some = wk && in;
        w1[i] = some ? pair(to_f(wk[e1 + 2 * i]), to_f(wk[e1 + 2 * i + 1])) : pair(1.f);
        w2[i] = some ? pair(to_f(wk[e2 + 2 * i]), to_f(wk[e2 + 2 * i + 1])) : pair(1.f);
        dw1[i] = dw2[i] = pair(0.f);
    }
    const int batches = (H + HEADS * U - 1) / (HEADS * U);
    Walk now(int64_t(block) * 8 + warp, int64_t(blocks) * 8, a.tokens, T_, batches), to = now;
    auto place_of = [&](const Walk &at) {
        return a.positions && at.left > 0 ? a.positions[at.b * a.ps[0] + at.t * a.ps[1]] : at.t;
    };
    // copies the unit `to`, whose position is `place`, and goes to the next one, whose position it loads
    int place = place_of(to);
    auto fetch = [&](int stage) -> bool {
        const bool live = a.R == 0 || (place >= 0 && place < a.rows);
        if (to.left > 0 && live) {
            unsigned char *at = ring + stage * kStageBytes<T, BWD>;
            if (a.R > 0) {
                const float *row = a.table + int64_t(place) * a.R;
                float *dst = reinterpret_cast<float *>(at);
                for (int e = 4 * lane; e < a.R; e += 128) copy16(dst + e, row + e);
            }
            T *x = reinterpret_cast<T *>(at + 1024) + sub * D;
            const int h0 = to.batch * U * HEADS + sub;
            const T *src = (const T *)r.x + (to.b * r.xs[0] + to.t * r.xs[1] + h0 * r.xs[2]);
            const T *gy = (const T *)r.gy + (to.b * r.gs[0] + to.t * r.gs[1] + h0 * r.gs[2]);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h0 - sub + u * HEADS >= H) break;
                if (h0 + u * HEADS < H) {
                    copy_head<T, G, VEC>(x + u * HEADS * D, src + u * HEADS * r.xs[2], D, g);
                    if (BWD) copy_head<T, G, VEC>(x + HALF + u * HEADS * D, gy + u * HEADS * r.gs[2], D, g);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        to.next(T_, batches);
        place = place_of(to);
        return live;
    };
    unsigned live = 0;  // of the units on their way, a bit for each: the oldest one lowest
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) live |= unsigned(fetch(i)) << i;
    int stage = 0;
    while (now.left > 0) {
        const int free = stage == 0 ? kStages - 1 : stage - 1;
        __syncwarp();  // it has been read
        live |= unsigned(fetch(free)) << (kStages - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        const unsigned char *at = ring + stage * kStageBytes<T, BWD>;
        float c[P] = {1.f, 1.f, 1.f, 1.f}, s[P] = {};
        if (turned && (live & 1u)) {
            const float *row = reinterpret_cast<const float *>(at) + P * g;
            load4(row, c);
            load4(row + half, s);
        }
        if (BWD) {
#pragma unroll
            for (int i = 0; i < P; ++i) s[i] = -s[i];
        }
        Turn<IL> turn;
        turn.set(c, s);
        const T *x = reinterpret_cast<const T *>(at + 1024) + sub * D;
        const int h0 = now.batch * U * HEADS + sub;
        T *out = (T *)r.out + ((int64_t(now.b) * T_ + now.t) * H + h0) * D;
        // all: every lane has elements of a head (no selects)
        auto work = [&](auto all) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (h0 - sub + u * HEADS >= H) break;
                const bool here = all.value || h0 + u * HEADS < H, some = all.value || (here && in && (live & 1u));
                f2 v1[2], v2[2], sq = pair(0.f);
                get4(x + u * HEADS * D + e1, some, v1), get4(x + u * HEADS * D + e2, some, v2);
#pragma unroll
                for (int i = 0; i < 2; ++i) sq = fma2(v1[i], v1[i], fma2(v2[i], v2[i], sq));
                const float2 q = both(sq);
                const float mean = group_sum<G>(q.x + q.y) * inv_d + a.eps;
                // (of no head: nothing, eps 0 too)
                const f2 rstd = pair(all.value || (here && (live & 1u)) ? rsqrtf(mean) : 0.f);
                if constexpr (!BWD) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) v1[i] = v1[i] * rstd * w1[i], v2[i] = v2[i] * rstd * w2[i];
                    turn(v1, v2);
                } else {
                    f2 g1[2], g2[2], d2 = pair(0.f);
                    get4(x + HALF + u * HEADS * D + e1, some, g1), get4(x + HALF + u * HEADS * D + e2, some, g2);
                    turn(g1, g2);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        v1[i] = v1[i] * rstd, v2[i] = v2[i] * rstd;
                        dw1[i] = fma2(g1[i], v1[i], dw1[i]), dw2[i] = fma2(g2[i], v2[i], dw2[i]);
                        g1[i] = g1[i] * w1[i], g2[i] = g2[i] * w2[i];
                        d2 = fma2(g1[i], v1[i], fma2(g2[i], v2[i], d2));
                    }
                    const float2 d = both(d2);
                    const f2 dot = pair(-inv_d * group_sum<G>(d.x + d.y));
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        v1[i] = rstd * fma2(dot, v1[i], g1[i]);
                        v2[i] = rstd * fma2(dot, v2[i], g2[i]);
                    }
                }
                if (!(here && in)) continue;
                if (!all.value && !(live & 1u)) v1[0] = v1[1] = v2[0] = v2[1] = pair(0.f);  // an empty row, whatever the weights
                put4<VEC>(out + u * HEADS * D + e1, v1);
                put4<VEC>(out + u * HEADS * D + e2, v2);
            }
        };
        if (D == 8 * G && H % HEADS == 0 && (live & 1u)) work(std::true_type());
        else work(std::false_type());
        now.next(T_, batches);
        live >>= 1;
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    __syncthreads();
    float(*red)[256] = reinterpret_cast<float(*)[256]>(smem);
    if constexpr (BWD) {
        // a block's sums: over the warp's heads, then over the warps
        auto block_sum = [&](const f2 (&d)[2], int e) {
            const float2 lo = both(d[0]), hi = both(d[1]);
            float v[P] = {lo.x, lo.y, hi.x, hi.y};
#pragma unroll
            for (int i = 0; i < P; ++i) {
#pragma unroll
                for (int m = G; m < 32; m *= 2) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m);
                if (sub == 0 && in) red[warp][e + i] = v[i];
            }
        };
        block_sum(dw1, e1);
        block_sum(dw2, e2);
        __syncthreads();
        if (int(threadIdx.x) < a.D) {
            float sum = red[0][threadIdx.x];
#pragma unroll
            for (int i = 1; i < 8; ++i) sum += red[i][threadIdx.x];
            part[int64_t(blockIdx.x) * a.D + threadIdx.x] = sum;
        }
    }
}

// dw[e] = the sum over the parts of its blocks, in a fixed order: 8 columns and 32 runs
// of blocks a thread block; the first D / 8 blocks the queries', the others the keys'
template <typename T>
__global__ void __launch_bounds__(256)
    qk_dw_kernel(const float *__restrict__ part, T *dwq, T *dwk, int first, int parts, int D) {
    __shared__ float red[32][9];
    const bool keys = int(blockIdx.x) >= D / 8;
    const int c = threadIdx.x & 7, k = threadIdx.x >> 3, col = (int(blockIdx.x) - (keys ? D / 8 : 0)) * 8;
    T *dw = keys ? dwk : dwq;
    griddep_wait();
    if (dw == nullptr) return;
    float s = 0.f;
    const int to = keys ? parts : first;
#pragma unroll 8
    for (int i = (keys ? first : 0) + k; i < to; i += 32) s += part[int64_t(i) * D + col + c];
    red[k][c] = s;
    __syncthreads();
    // warp j adds up column j
    const int lane = threadIdx.x & 31, j = threadIdx.x >> 5;
    s = red[lane][j];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
    if (lane == 0) dw[col + j] = from_f<T>(s);
}

// Lanes of a head: a power of two, at least 4, of 8 elements each
int lanes_of(int D) {
    int g = 4;
    while (g * 8 < D) g *= 2;
    return g;
}

// Blocks of the queries and of the keys, in the ratio of their heads: as many as are
// resident, fewer for fewer tokens.
struct Grid {
    int q, k;
};
template <typename T, bool BWD>
Grid grid_of(int64_t tokens, int Hq, int Hk, int D) {
    const int64_t most = 152 * kBlocksPerSm<T>, once = 32 / lanes_of(D) * kOnce<T, BWD>;
    auto need = [&](int H) { return (min64(tokens, int64_t(1) << 40) * ((H + once - 1) / once) + 7) / 8; };
    int64_t q = need(Hq), k = need(Hk);
    if (q + k > most) {
        const int64_t all = most * Hq / (int64_t(Hq) + Hk);
        const int64_t mq = all < 1 ? 1 : all > most - 1 ? most - 1 : all;
        q = Hq == 0 ? 0 : Hk == 0 ? most : min64(q, mq);
        k = Hk == 0 ? 0 : min64(k, most - q);
    }
    return {int(q), int(k)};
}

template <int N>
using Int = std::integral_constant<int, N>;

template <typename T, bool BWD>
cudaError_t go(Args &a, bool interleaved, float *part, int *blocks, cudaStream_t s) {
    // copies of 16 bytes where all tensors allow them
    constexpr int V = kVec<T>;
    bool vec = true;
    for (const Rows &r : a.r) {
        if (r.H == 0) continue;
        for (const void *p : {r.x, r.gy, (const void *)r.out}) vec = vec && reinterpret_cast<uintptr_t>(p) % 16 == 0;
        for (int i = 0; i < 3; ++i) vec = vec && r.xs[i] % V == 0 && r.gs[i] % V == 0;
    }
    const Grid grid = grid_of<T, BWD>(a.tokens, a.r[0].H, a.r[1].H, a.D);
    a.first = grid.q;
    *blocks = grid.q + grid.k;
    auto run = [&](auto g, auto v, auto il) {
        auto *fn = qk_norm_kernel<T, g.value, v.value, il.value, BWD>;
        constexpr int bytes = 8 * kStages * kStageBytes<T, BWD>;
        const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(fn), bytes);
        if (e != cudaSuccess) return e;
        fn<<<unsigned(grid.q + grid.k), 256, bytes, s>>>(a, part);
        return cudaGetLastError();
    };
    auto lanes = [&](auto v, auto il) {
        const int g = lanes_of(a.D);
        if (g == 4) return run(Int<4>(), v, il);
        if (g == 8) return run(Int<8>(), v, il);
        if (g == 16) return run(Int<16>(), v, il);
        return run(Int<32>(), v, il);
    };
    auto pairs = [&](auto v) { return interleaved ? lanes(v, std::true_type()) : lanes(v, std::false_type()); };
    return vec ? pairs(std::true_type()) : pairs(std::false_type());
}

Args args_of(const mgs_qk_norm_shape &sh, const void *q, const void *k, const void *qw, const void *kw,
             const void *gq, const void *gk, const float *table, const int32_t *positions, void *oq, void *ok) {
    Args a = {};
    a.r[0] = {q, qw, gq, oq, {}, {}, int(sh.Hq)}, a.r[1] = {k, kw, gk, ok, {}, {}, int(sh.Hk)};
    for (int i = 0; i < 3; ++i) {
        a.r[0].xs[i] = sh.q_stride[i], a.r[1].xs[i] = sh.k_stride[i];
        if (gq || gk) a.r[0].gs[i] = sh.gq_stride[i], a.r[1].gs[i] = sh.gk_stride[i];
    }
    a.table = table, a.positions = positions, a.ps[0] = sh.pos_stride[0], a.ps[1] = sh.pos_stride[1];
    a.rows = sh.positions, a.tokens = sh.B * sh.T, a.T = sh.T, a.D = sh.D, a.R = sh.rotary, a.eps = sh.eps;
    return a;
}

}  // namespace

cudaError_t launch_qk_norm_fwd(const mgs_qk_norm_shape &sh, const void *q, const void *k, const void *qw,
                               const void *kw, const float *table, const int32_t *positions, void *yq, void *yk,
                               cudaStream_t s) {
    Args a = args_of(sh, q, k, qw, kw, nullptr, nullptr, table, positions, yq, yk);
    int blocks;
    return sh.dtype == MGS_BF16 ? go<bf16, false>(a, sh.interleaved, nullptr, &blocks, s)
                                : go<float, false>(a, sh.interleaved, nullptr, &blocks, s);
}

size_t qk_norm_bwd_workspace_bytes(const mgs_qk_norm_shape &sh) {
    const int64_t tokens = sh.B * sh.T;
    const Grid g = sh.dtype == MGS_BF16 ? grid_of<bf16, true>(tokens, int(sh.Hq), int(sh.Hk), sh.D)
                                        : grid_of<float, true>(tokens, int(sh.Hq), int(sh.Hk), sh.D);
    return size_t(g.q + g.k) * size_t(sh.D) * 4;
}

cudaError_t launch_qk_norm_bwd(const mgs_qk_norm_shape &sh, const void *q, const void *k, const void *qw,
                               const void *kw, const void *gq, const void *gk, const float *table,
                               const int32_t *positions, void *dq, void *dk, void *dqw, void *dkw, void *ws,
                               cudaStream_t s) {
    Args a = args_of(sh, q, k, qw, kw, gq, gk, table, positions, dq, dk);
    float *part = static_cast<float *>(ws);
    int blocks;
    const cudaError_t e = sh.dtype == MGS_BF16 ? go<bf16, true>(a, sh.interleaved, part, &blocks, s)
                                               : go<float, true>(a, sh.interleaved, part, &blocks, s);
    if (e != cudaSuccess || (dqw == nullptr && dkw == nullptr)) return e;
    return sh.dtype == MGS_BF16 ? launch_next(qk_dw_kernel<bf16>, unsigned(2 * sh.D / 8), 256, 0, s, true, part,
                                              (bf16 *)dqw, (bf16 *)dkw, a.first, blocks, sh.D)
                                : launch_next(qk_dw_kernel<float>, unsigned(2 * sh.D / 8), 256, 0, s, true, part,
                                              (float *)dqw, (float *)dkw, a.first, blocks, sh.D);
}

}  // namespace mgs
