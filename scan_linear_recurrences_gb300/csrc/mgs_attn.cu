// Linear attention with a decay for each head.  Per (batch, head), state S
// (D x D, key index first):
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t.
// With R_t = dL/dS_t = e^{g_{t+1}} R_{t+1} + scale q_t do_t^T the gradients are
//   dq_t = scale S_t do_t,  dk_t = R_t v_t,  dv_t = R_t^T k_t,
// each of which is the same map of other tensors (F(q, k, v) for the map):
//   dq = F(do, v, k) on S^T;  dk = F(v, do, q) and dv = F(k, q, do) in reverse
// time.  One walking kernel therefore serves attention and its three
// gradients (AttnWalk).  The decay's gradient dg_t = <R_t, e^{g_t} S_{t-1}>
// obeys dg_t = dg_{t+1} + <q_t, dq_t> - <k_t, dk_t>; summing that over a long
// sequence in fp32 would lose digits, so the walks leave S and R at the end of
// every span of steps and the sum restarts there from <R, S>.
//
// Few (batch, head) lanes and a long sequence: time is cut into segments; a
// state-only walk gives each segment's own state, a short scan joins them, and
// the full walk then starts every segment from its state.
#include "mgs_lm.h"
#include "mgs_num.cuh"

namespace mgs {
namespace {

constexpr int TS = 16;  // time steps staged in shared memory at once

// The recurrence itself, in fp32 (SIMT).  A block owns one lane's (segment
// of) time with the whole D x D state in registers: a thread holds 32 key
// rows of one column, P = D / 32 neighbouring threads share a column.  Per
// step and thread 32 x 4 fp32 operations: bound by the fp32 pipes (64 lanes of
// 1024 steps, heads of 128 in fp32: 684 us, where the tensor-core walk takes
// 113).  For tensors that no tensor map describes.
template <typename TI, int D, bool STATE_ONLY>
__global__ void __launch_bounds__(D *D / 32) attn_rec_kernel(const __grid_constant__ AttnSet set) {
    constexpr int P = D / 32, NT = D * D / 32, V4 = TS * D / 4, NL = V4 / NT;
    static_assert(NL >= 1 && V4 % NT == 0, "whole vectors a thread");
    __shared__ __align__(16) float sq[TS * D], sk[TS * D], sv[TS * D];
    __shared__ float2 sa[TS];  // e^g in two parts: its rounding would be that of every step of a fixed decay
    __shared__ float sg[TS];
    const AttnWalk &w = set.w[blockIdx.y];
    const int nseg = set.nseg;
    const int64_t lane = blockIdx.x / nseg;
    const int seg = int(blockIdx.x % nseg);
    const int b = int(lane / set.H), h = int(lane % set.H);
    if (STATE_ONLY && seg == (w.rev ? 0 : nseg - 1)) return;  // nothing starts from this segment's state
    const int64_t t0 = seg * set.seg_len, t1 = min64(set.T, t0 + set.seg_len);
    const int tid = threadIdx.x, part = tid % P, col = tid / P;
    const TI *q = static_cast<const TI *>(w.q) + b * w.qs[0] + (h / w.qdiv) * w.qs[2];
    const TI *k = static_cast<const TI *>(w.k) + b * w.ks[0] + (h / w.kdiv) * w.ks[2];
    const TI *v = static_cast<const TI *>(w.v) + b * w.vs[0] + (h / w.vdiv) * w.vs[2];
    const float *g = set.g + b * set.gs[0] + h * set.gs[2];

    // row of state element i of this thread
    auto row = [&](int i) { return 4 * (part + P * (i >> 2)) + (i & 3); };
    float s[32];
    {
        const float *in = nullptr;
        bool tr = false;
        if (!STATE_ONLY) {
            if (nseg > 1)
                in = w.seg_in + (lane * nseg + seg) * D * D;
            else if (w.s_in)
                in = w.s_in + lane * D * D, tr = w.s_in_t;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) s[i] = in == nullptr ? 0.f : tr ? in[col * D + row(i)] : in[row(i) * D + col];
    }
    auto put_state = [&](float *to, bool tr) {
#pragma unroll
        for (int i = 0; i < 32; ++i) to[tr ? col * D + row(i) : row(i) * D + col] = s[i];
    };

    float rq[NL][4], rk[NL][4], rv[NL][4], rg = 0.f;
    auto fetch = [&](int64_t base, int n) {
#pragma unroll
        for (int l = 0; l < NL; ++l) {
            const int e = tid + l * NT, u = e / (D / 4), c = 4 * (e % (D / 4));
            if (u < n) {
                if (!STATE_ONLY) load4(q + (base + u) * w.qs[1] + c, rq[l]);
                load4(k + (base + u) * w.ks[1] + c, rk[l]);
                load4(v + (base + u) * w.vs[1] + c, rv[l]);
            }
        }
        if (tid < n) rg = g[(base + tid) * set.gs[1]];
    };
    auto stage = [&](int n) {
#pragma unroll
        for (int l = 0; l < NL; ++l) {
            const int e = tid + l * NT;
            if (e / (D / 4) < n) {
                if (!STATE_ONLY) store4(sq + 4 * e, rq[l]);
                store4(sk + 4 * e, rk[l]);
                store4(sv + 4 * e, rv[l]);
            }
        }
        if (tid < n) exp_two(rg, sa[tid].x, sa[tid].y), sg[tid] = rg;
    };

    double total = 0.0;  // thread 0, state-only: the segment's sum of g
    // tiles are [base, base + n) with base a multiple of TS, walked up or down
    int64_t base = w.rev ? (t1 - 1) / TS * TS : t0;
    int n = int(min64(TS, t1 - base));
    if (t0 < t1) fetch(base, n);
    while (base >= t0 && base < t1) {
        stage(n);
        __syncthreads();
        const int64_t nbase = w.rev ? base - TS : base + TS;
        const int nn = int(min64(TS, t1 - nbase));
        if (nbase >= t0 && nbase < t1) fetch(nbase, nn);
        const int64_t end = base + n;
        const bool keep = !STATE_ONLY && w.ckpt && (end % set.span == 0 || end == set.T) && (end - 1) / set.span < set.kept;
        if (keep && w.rev)
            put_state(w.ckpt + (lane * set.spans + (end - 1) / set.span) * D * D, false);
        if (STATE_ONLY && tid == 0)
            for (int u = 0; u < n; ++u) total += double(sg[u]);
        float2 prev = make_float2(1.f, 0.f);  // reverse: the decay of step t + 1, applied as step t is added
        for (int i = 0; i < n; ++i) {
            const int u = w.rev ? n - 1 - i : i;
            const float2 a = w.rev ? prev : sa[u];
            prev = sa[u];
            const float vc = sv[u * D + col] * w.kv_scale;
            const float4 *k4 = reinterpret_cast<const float4 *>(sk + u * D) + part;
            const float4 *q4 = reinterpret_cast<const float4 *>(sq + u * D) + part;
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                const float4 kk = k4[c * P];
                s[4 * c + 0] = fmaf(a.x, s[4 * c + 0], fmaf(a.y, s[4 * c + 0], kk.x * vc));
                s[4 * c + 1] = fmaf(a.x, s[4 * c + 1], fmaf(a.y, s[4 * c + 1], kk.y * vc));
                s[4 * c + 2] = fmaf(a.x, s[4 * c + 2], fmaf(a.y, s[4 * c + 2], kk.z * vc));
                s[4 * c + 3] = fmaf(a.x, s[4 * c + 3], fmaf(a.y, s[4 * c + 3], kk.w * vc));
                if (!STATE_ONLY) {
                    const float4 qq = q4[c * P];
                    acc[0] = fmaf(qq.x, s[4 * c + 0], acc[0]);
                    acc[1] = fmaf(qq.y, s[4 * c + 1], acc[1]);
                    acc[2] = fmaf(qq.z, s[4 * c + 2], acc[2]);
                    acc[3] = fmaf(qq.w, s[4 * c + 3], acc[3]);
                }
            }
            if (!STATE_ONLY) {
                float o = (acc[0] + acc[1]) + (acc[2] + acc[3]);
#pragma unroll
                for (int m = 1; m < P; m <<= 1) o += __shfl_xor_sync(0xffffffffu, o, m);
                // the column's own v of this step was read above by all P threads of the column
                __syncwarp();
                if (part == 0) sv[u * D + col] = o * w.o_scale;
            }
        }
        if (w.rev) {
#pragma unroll
            for (int i = 0; i < 32; ++i) s[i] = fmaf(prev.x, s[i], prev.y * s[i]);
        }
        __syncthreads();
        if (!STATE_ONLY) {
            // the tile's outputs (left in sv) to memory, and their products with x
#pragma unroll
            for (int l = 0; l < NL; ++l) {
                const int e = tid + l * NT, u = e / (D / 4), c = 4 * (e % (D / 4));
                float o[4] = {0.f, 0.f, 0.f, 0.f}, dot = 0.f;
                if (u < n) {
                    load4(sv + 4 * e, o);
                    const int64_t at = b * w.os[0] + (base + u) * w.os[1] + h * w.os[2] + c;
                    if (w.out_f32)
                        store4(static_cast<float *>(w.out) + at, o);
                    else
                        store4(static_cast<TI *>(w.out) + at, o);
                    if (w.row_dot) {
                        float x[4];
                        load4(static_cast<const TI *>(w.x) + b * w.xs[0] + (base + u) * w.xs[1] +
                                  (h / w.xdiv) * w.xs[2] + c,
                              x);
                        dot = (o[0] * x[0] + o[1] * x[1]) + (o[2] * x[2] + o[3] * x[3]);
                    }
                }
                if (w.row_dot) {
#pragma unroll
                    for (int m = 1; m < D / 4; m <<= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
                    if (u < n && c == 0) w.row_dot[lane * set.T + base + u] = dot;
                }
            }
            if (keep && !w.rev)
                put_state(w.ckpt + (lane * set.spans + (end - 1) / set.span) * D * D, false);
            __syncthreads();
        }
        base = nbase;
        n = nn;
    }
    if (STATE_ONLY) {
        float *to = w.seg_out + (lane * nseg + seg) * D * D;
        put_state(to, false);
        if (tid == 0) w.seg_out[int64_t(set.B) * set.H * nseg * D * D + lane * nseg + seg] = float(total);
    } else if (w.s_out && seg == (w.rev ? 0 : nseg - 1)) {
        put_state(w.s_out + lane * D * D, false);
    }
}

// Joins the segments' own states into the state at each segment's start (in
// place): elementwise over the D x D entries, a thread a run of 4.  The
// segments' states are read eight at a time, before any of them is replaced: a
// chain of single reads would be as many trips to memory as there are segments
// (44 us for 9 segments of 16 lanes, against 5).
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnSet set) {
    constexpr int N = 8;
    const AttnWalk &w = set.w[blockIdx.z];
    const int64_t lane = blockIdx.y;
    const int e = 4 * int(blockIdx.x * blockDim.x + threadIdx.x);
    const int nseg = set.nseg;
    griddep_launch();
    griddep_wait();
    float *st = w.seg_out + lane * nseg * D * D + e;
    const float *total = w.seg_out + int64_t(set.B) * set.H * nseg * D * D + lane * nseg;
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    if (w.s_in) {
        const float *in = w.s_in + lane * D * D;
        if (!w.s_in_t) {
            load4(in + e, s);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = in[((e + i) % D) * D + (e + i) / D];
        }
    }
    for (int i0 = 0; i0 < nseg; i0 += N) {
        float own[N][4], a[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int i = i0 + j, seg = w.rev ? nseg - 1 - i : i;
            if (i + 1 < nseg) {  // nothing follows from the last one's state
                load4(st + int64_t(seg) * D * D, own[j]);
                a[j] = total[seg];
            }
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int i = i0 + j, seg = w.rev ? nseg - 1 - i : i;
            if (i >= nseg) break;
            store4(st + int64_t(seg) * D * D, s);
            if (i + 1 < nseg) {
                const float f = expf(a[j]);
#pragma unroll
                for (int c = 0; c < 4; ++c) s[c] = fmaf(f, s[c], own[j][c]);
            }
        }
    }
}

// The sum over a block of 256 threads, as a pair.
__device__ __forceinline__ float2 block_sum(float2 x, float2 *red) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1)
        add2(x.x, x.y, __shfl_xor_sync(0xffffffffu, x.x, m), __shfl_xor_sync(0xffffffffu, x.y, m));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    float2 t = red[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) add2(t.x, t.y, red[i].x, red[i].y);
    return t;
}

// dg over one span: dg_t = <R_e, S_e> + sum_{t <= s < e} (<q_s, dq_s> - <k_s, dk_s>),
// e the span's end.  With a decay of one number a head, the span's sum of dg goes
// to part[lane][span] instead.  These sums cancel (of a fixed decay's, all but one
// part in a hundred), so they are of pairs of fp32.  Bound by the reads of S and R
// (128 lanes of 8 spans, heads of 128: 117 MB in 30 us).
__global__ void __launch_bounds__(256)
    attn_dg_kernel(const float *__restrict__ u, const float *__restrict__ w, int parts, const float *__restrict__ ckS,
                   const float *__restrict__ ckR, float *__restrict__ dg, float2 *__restrict__ part, int64_t T,
                   int64_t H, int spans, int kept, int span_steps, int DD) {
    __shared__ float2 red[8], scan[8];
    constexpr int NT = 256;  // threads, each with one or two of the span's steps
    griddep_wait();
    const int64_t lane = blockIdx.x / spans;
    const int span = int(blockIdx.x % spans), tid = threadIdx.x, per = span_steps > NT ? 2 : 1;
    const int64_t b = lane / H, h = lane % H;
    const int64_t t0 = int64_t(span) * span_steps;
    const int n = int(min64(span_steps, T - t0));
    float2 tail = make_float2(0.f, 0.f);
    if (span < kept) {
        const float *a = ckS + (lane * spans + span) * DD, *c = ckR + (lane * spans + span) * DD;
        float acc = 0.f;
        for (int e0 = 4 * tid; e0 < DD; e0 += 16 * NT) {  // DD is a multiple of 4096: four pieces at a time
            float x[4][4], y[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) load4(a + e0 + 4 * NT * j, x[j]), load4(c + e0 + 4 * NT * j, y[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc += (x[j][0] * y[j][0] + x[j][1] * y[j][1]) + (x[j][2] * y[j][2] + x[j][3] * y[j][3]);
        }
        tail = block_sum(make_float2(acc, 0.f), red);
    }
    const int64_t all = int64_t(gridDim.x) / spans * T;  // of one part
    // suffix sums: thread i holds steps per i .. per i + per - 1
    float2 d[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
    for (int p = 0; p < parts; ++p) {
        float x[2], y[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = per * tid + i;
            const int64_t at = lane * T + t0 + t + p * all;
            x[i] = i < per && t < n ? u[at] : 0.f;
            y[i] = i < per && t < n ? w[at] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) add2(d[i].x, d[i].y, x[i], 0.f), add2(d[i].x, d[i].y, -y[i], 0.f);
    }
    add2(d[0].x, d[0].y, d[1].x, d[1].y);
    float2 suf = d[0];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const float oh = __shfl_down_sync(0xffffffffu, suf.x, m), ol = __shfl_down_sync(0xffffffffu, suf.y, m);
        if ((tid & 31) + m < 32) add2(suf.x, suf.y, oh, ol);
    }
    __syncthreads();
    if ((tid & 31) == 0) scan[tid >> 5] = suf;
    __syncthreads();
    const float nh = __shfl_down_sync(0xffffffffu, suf.x, 1), nl = __shfl_down_sync(0xffffffffu, suf.y, 1);
    float2 after = tail, sum = make_float2(0.f, 0.f);
    if ((tid & 31) != 31) add2(after.x, after.y, nh, nl);
    for (int i = (tid >> 5) + 1; i < NT / 32; ++i) add2(after.x, after.y, scan[i].x, scan[i].y);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int t = per * tid + i;
        if (i >= per || t >= n) continue;
        float2 x = d[i];
        add2(x.x, x.y, after.x, after.y);
        add2(sum.x, sum.y, x.x, x.y);
        if (dg) dg[(b * T + t0 + t) * H + h] = x.x;
    }
    if (part) {
        sum = block_sum(sum, red);
        if (tid == 0) part[lane * spans + span] = sum;
    }
}

// dg[h] = sum over batch and spans, in a fixed order: a few thousand numbers, 3 us
__global__ void __launch_bounds__(256)
    attn_dg_fixed_kernel(const float2 *__restrict__ part, float *__restrict__ dg, int64_t B, int64_t H, int spans) {
    __shared__ float2 red[8];
    const int64_t h = blockIdx.x;
    float2 acc = make_float2(0.f, 0.f);
    for (int64_t i = threadIdx.x; i < B * spans; i += blockDim.x) {
        const float2 x = part[((i / spans) * H + h) * spans + i % spans];
        add2(acc.x, acc.y, x.x, x.y);
    }
    acc = block_sum(acc, red);
    if (threadIdx.x == 0) dg[h] = acc.x;
}

// out[row][hk][D] = sum of the group's heads of in[row][H][D].  Bound by memory.
template <typename TO>
__global__ void attn_group_sum_kernel(const float *__restrict__ in, TO *__restrict__ out, int64_t n4, int D4,
                                      int64_t Hk, int group) {
    for (int64_t e = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; e < n4; e += int64_t(gridDim.x) * blockDim.x) {
        const int64_t rh = e / D4;
        const int c = int(e - rh * D4);
        float s[4] = {0.f, 0.f, 0.f, 0.f}, x[4];
        for (int i = 0; i < group; ++i) {
            load4(in + 4 * ((rh * group + i) * D4 + c), x);
#pragma unroll
            for (int j = 0; j < 4; ++j) s[j] += x[j];
        }
        store4(out + 4 * e, s);
    }
}

// fp32 as three bf16 tensors: x = a + b + c, each the rest rounded (24 bits).
// Bound by memory: 10 bytes an element (q, k, v of 128 x 1024 x 64: 39 us, 6.3 TB/s).
struct SplitSet {
    const float *in[4];
    bf16 *out[4];
    int64_t st[4][3];
    int heads[4];
    int64_t B, T;
};
template <int D>
__global__ void __launch_bounds__(256) attn_split_kernel(const __grid_constant__ SplitSet set) {
    griddep_launch();
    const int which = blockIdx.y, heads = set.heads[which];
    const int64_t rows = set.B * set.T * heads, n4 = rows * (D / 4), plane = rows * D;
    const float *in = set.in[which];
    bf16 *out = set.out[which];
    for (int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x; e < n4; e += int64_t(gridDim.x) * 256) {
        const int64_t row = e / (D / 4), bt = row / heads, b = bt / set.T;
        const int c = 4 * int(e - row * (D / 4));
        const float4 x = *reinterpret_cast<const float4 *>(in + b * set.st[which][0] + (bt - b * set.T) * set.st[which][1] +
                                                           (row - bt * heads) * set.st[which][2] + c);
        float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int m = 0; m < 3; ++m) {
            const uint2 t = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            *reinterpret_cast<uint2 *>(out + m * plane + 4 * e) = t;
            v[0] -= bf_lo(t.x), v[1] -= bf_hi(t.x), v[2] -= bf_lo(t.y), v[3] -= bf_hi(t.y);
        }
    }
}

// One token.  A block holds 32 columns of one head's state: 8 threads across
// (float4), 32 groups of D / 32 rows; the rows' products with q are summed in
// shared memory.  Bound by the state's bytes, read and written once (384 users
// of 16 heads of 128: 806 MB in 132 us, 6.1 TB/s; 16 heads of one user: 2.5 us).
template <typename TI, int D>
__global__ void __launch_bounds__(256)
    attn_step_kernel(const TI *__restrict__ q, const TI *__restrict__ k, const TI *__restrict__ v,
                     const float *__restrict__ g, float *__restrict__ S, const int32_t *__restrict__ slots,
                     TI *__restrict__ o, mgs_attention_shape sh, int64_t nslots) {
    constexpr int R = D / 32;
    __shared__ float red[32][33];
    const int64_t lane = blockIdx.x / (D / 32);
    const int c0 = 32 * int(blockIdx.x % (D / 32));
    const int64_t b = lane / sh.H, h = lane % sh.H, hk = h / (sh.H / sh.Hk);
    const int tid = threadIdx.x, cx = 4 * (tid & 7), rg = tid >> 3;
    TI *out = o + (b * sh.H + h) * D + c0;
    const int64_t slot = slots ? slots[b] : b;
    if (slot < 0 || slot >= nslots) {
        if (tid < 32) out[tid] = from_f<TI>(0.f);
        return;
    }
    float *st = S + (slot * sh.H + h) * D * D + c0 + cx;
    float4 x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = *reinterpret_cast<const float4 *>(st + (rg + 32 * r) * D);
    const float a = expf(sh.fixed_decay ? g[h] : g[b * sh.g_stride[0] + h * sh.g_stride[2]]);
    float vv[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
    load4(v + b * sh.v_stride[0] + h * sh.v_stride[2] + c0 + cx, vv);
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float kk = to_f(k[b * sh.k_stride[0] + hk * sh.k_stride[2] + rg + 32 * r]);
        const float qq = to_f(q[b * sh.q_stride[0] + hk * sh.q_stride[2] + rg + 32 * r]);
        x[r].x = fmaf(kk, vv[0], a * x[r].x);
        x[r].y = fmaf(kk, vv[1], a * x[r].y);
        x[r].z = fmaf(kk, vv[2], a * x[r].z);
        x[r].w = fmaf(kk, vv[3], a * x[r].w);
        *reinterpret_cast<float4 *>(st + (rg + 32 * r) * D) = x[r];
        acc[0] = fmaf(qq, x[r].x, acc[0]);
        acc[1] = fmaf(qq, x[r].y, acc[1]);
        acc[2] = fmaf(qq, x[r].z, acc[2]);
        acc[3] = fmaf(qq, x[r].w, acc[3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[rg][cx + i] = acc[i];
    __syncthreads();
    // 8 threads a column, 4 rows each
    const int c = tid >> 3, r0 = tid & 7;
    float s = (red[r0][c] + red[r0 + 8][c]) + (red[r0 + 16][c] + red[r0 + 24][c]);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    s += __shfl_xor_sync(0xffffffffu, s, 4);
    if (r0 == 0) out[c] = from_f<TI>(s * sh.scale);
}

// ---------------------------------------------------------------- host side
// The tensor-core walk takes bf16 tensors whose steps, heads and batch rows lie
// apart in memory (a TMA tensor map has no zero strides), and fp32.
bool mma_takes(const mgs_attention_shape &sh, bool backward) {
    auto apart = [&](const int64_t (&st)[3], int64_t heads) {
        return (sh.B == 1 || st[0] > 0) && (sh.T == 1 || st[1] > 0) && (heads == 1 || st[2] > 0);
    };
    const bool qk = apart(sh.q_stride, sh.Hk) && apart(sh.k_stride, sh.Hk);
    // fp32 is read through its terms' tensors, but for the products of q with dq and k with dk
    if (sh.dtype != MGS_BF16) return qk || !backward;
    return qk && apart(sh.v_stride, sh.H) && (!backward || apart(sh.do_stride, sh.H));
}

// Steps over which the decay's gradient is summed between exact restarts, whole
// chunks and at most 512.  The error grows with them, the states to be kept shrink
// (the gradients of 128 lanes of 4096 steps, heads of 128 in bf16: 517 us with 1024,
// 523 with 512, 556 with 256; dg's error up to 1.6e-6, 9e-7, 6e-7; in fp32, 64 lanes
// of 1024 steps: 270 with 512, 278 with 256, dg's error 7e-7 with 256).  A decay of
// one number a head has the sum of a whole batch's, which cancels further: chunk by
// chunk (8 x 1000 steps, 8 heads of 128 in bf16: 4.4e-6, against 8.8e-6 with 256 and
// 4.3e-5 with 1024).
constexpr int kSpanF32 = 256, kSpanBF16 = 512, kSpanFixed = 128;

struct Plan {
    int64_t lanes, chunks, seg_len;
    int nseg, spans, parts, span;
    bool mma;
};
Plan plan_of(const mgs_attention_shape &sh, int walks) {
    Plan p;
    p.mma = mma_takes(sh, walks == 3);
    const bool f32 = sh.dtype == MGS_F32;
    p.parts = !p.mma ? 1 : (sh.D == 128 ? 2 : 1) * (f32 ? 2 : 1);  // of a head's row products, one a warp
    p.lanes = sh.B * sh.H;
    p.chunks = (sh.T + kAttnChunk - 1) / kAttnChunk;
    // Segments of the time axis: as many as fill the 152 SMs with blocks (one
    // block to an SM for the tensor-core walk; the SIMT one wants more warps).
    // (two heads of 64 in bf16 share a block; a head of 128 in fp32 takes two)
    const int64_t units = !p.mma || (sh.D == 128) != f32 ? p.lanes : f32 ? 2 * p.lanes : sh.B * ((sh.H + 1) / 2);
    const int64_t want = 152 * (p.mma || sh.D == 128 ? 1 : 4);
    int64_t n = units * walks > 0 ? want / (units * walks) : 1;
    if (n > p.chunks) n = p.chunks;
    // They cost a state-only walk (half as long as a full one; nearly as long in
    // the SIMT kernel, which is cut in three or more only) and two more launches,
    // of about four chunks' time together (13 chunks in 5 segments, 30 blocks
    // each: 41 us against 66 in one).
    const int64_t len = n > 0 ? (p.chunks + n - 1) / n : p.chunks;
    if (n < (p.mma ? 2 : 3) || 3 * len + 8 >= 2 * p.chunks) n = 1;
    p.seg_len = (p.chunks + n - 1) / n * kAttnChunk;
    if (p.seg_len < kAttnChunk) p.seg_len = kAttnChunk;
    p.nseg = int((sh.T + p.seg_len - 1) / p.seg_len);
    if (p.nseg < 1) p.nseg = 1;
    p.span = sh.fixed_decay ? kSpanFixed : f32 ? kSpanF32 : kSpanBF16;
    p.spans = int((sh.T + p.span - 1) / p.span);
    return p;
}

size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// fp32 for the tensor cores: a tensor's three terms
size_t split_bytes(const mgs_attention_shape &sh, const Plan &p, int64_t heads) {
    return p.mma && sh.dtype == MGS_F32 ? up256(size_t(sh.B) * sh.T * heads * sh.D * 6) : 0;
}
size_t seg_bytes(const Plan &p, int D) {  // one walk's segment states and their sums of g
    return p.nseg > 1 ? up256(size_t(p.lanes) * p.nseg * (size_t(D) * D + 1) * 4) : 0;
}

// Hands out consecutive 256-byte aligned parts of the workspace.
struct Carve {
    char *p;
    template <typename T>
    T *take(size_t bytes) {
        T *r = reinterpret_cast<T *>(p);
        p += up256(bytes);
        return r;
    }
};

void copy3(int64_t (&to)[3], const int64_t (&from)[3]) {
    for (int i = 0; i < 3; ++i) to[i] = from[i];
}
void dense(int64_t (&st)[3], int64_t T, int64_t H, int64_t D) { st[0] = T * H * D, st[1] = H * D, st[2] = D; }

AttnSet set_of(const mgs_attention_shape &sh, const Plan &p, const float *g, const DevCtl &ctl) {
    AttnSet s = {};
    s.g = g;
    if (sh.fixed_decay)
        s.gs[0] = 0, s.gs[1] = 0, s.gs[2] = 1;
    else
        copy3(s.gs, sh.g_stride);
    s.B = sh.B, s.T = sh.T, s.H = sh.H;
    s.seg_len = p.seg_len, s.nseg = p.nseg, s.spans = p.spans, s.span = p.span;
    s.ctl = ctl;
    s.tries = uint32_t(min64(int64_t(ctl.timeout_ns / 40) + 1000, 0x7fffffff));
    for (auto &w : s.w) w.qdiv = w.kdiv = w.vdiv = w.xdiv = 1, w.o_scale = w.kv_scale = 1.f;
    return s;
}

// The terms of fp32 tensors, in the workspace; what the walks read of the others stays.
struct Splitter {
    const mgs_attention_shape &sh;
    const Plan &p;
    Carve &ws;
    SplitSet set = {};
    int n = 0;
    // p, its strides and, for fp32, their replacement
    const void *take(const void *in, const int64_t (&st)[3], int64_t heads, int64_t (&to)[3]) {
        copy3(to, st);
        const size_t bytes = split_bytes(sh, p, heads);
        if (bytes == 0) return in;
        set.in[n] = static_cast<const float *>(in);
        set.out[n] = ws.take<bf16>(bytes);
        copy3(set.st[n], st);
        set.heads[n] = int(heads);
        dense(to, sh.T, heads, sh.D);
        return set.out[n++];
    }
    cudaError_t run(cudaStream_t s) {
        if (n == 0) return cudaSuccess;
        set.B = sh.B, set.T = sh.T;
        const int64_t most = sh.B * sh.T * sh.H * (sh.D / 4);
        const dim3 grid(unsigned(min64((most + 255) / 256, 152 * 16)), unsigned(n));
        sh.D == 64 ? attn_split_kernel<64><<<grid, 256, 0, s>>>(set) : attn_split_kernel<128><<<grid, 256, 0, s>>>(set);
        return cudaGetLastError();
    }
};

cudaError_t run_walks(AttnSet &set, int walks, const mgs_attention_shape &sh, const Plan &p, Carve &ws,
                      cudaStream_t s) {
    cudaError_t e;
    // fp32 has three terms everywhere.  In bf16 the first two of the gradients'
    // walks feed the decay's, whose sums want every digit of fp32; of dv, and of the
    // attention itself, nothing but the rounding to the type follows: two.  dv's walk shares no tensor with
    // those two and fills the SMs that they leave (5 x 1537 steps, 12 heads of
    // 64: 173 us, one after the other 243).
    auto walk = [&](bool state_only) {
        if (!p.mma) return launch_attn_rec(set, walks, sh.D, sh.dtype, state_only, s);
        const bool early = !state_only && p.nseg > 1;  // after attn_join
        if (sh.dtype == MGS_F32) return launch_attn_mma(set, 0, walks, sh.D, sh.dtype, 3, state_only, true, false, s);
        if (walks == 1 || state_only) return launch_attn_mma(set, 0, walks, sh.D, sh.dtype, 2, state_only, early, false, s);
        const cudaError_t e = launch_attn_mma(set, 0, 2, sh.D, sh.dtype, 3, false, early, false, s);
        return e != cudaSuccess ? e : launch_attn_mma(set, 2, 1, sh.D, sh.dtype, 2, false, false, true, s);
    };
    if (set.nseg > 1) {
        for (int i = 0; i < walks; ++i) set.w[i].seg_in = set.w[i].seg_out = ws.take<float>(seg_bytes(p, sh.D));
        if ((e = walk(true)) != cudaSuccess) return e;
        const dim3 grid(unsigned(sh.D * sh.D / 1024), unsigned(sh.B * sh.H), unsigned(walks));
        auto *join = sh.D == 64 ? attn_join_kernel<64> : attn_join_kernel<128>;
        if ((e = launch_next(join, grid, 256, 0, s, p.mma, set)) != cudaSuccess) return e;
    }
    return walk(false);
}

}  // namespace

template <typename TI, int D>
static void rec_go(const AttnSet &set, int nwalks, bool state_only, cudaStream_t s) {
    const dim3 grid(unsigned(set.B * set.H * set.nseg), unsigned(nwalks));
    if (state_only)
        attn_rec_kernel<TI, D, true><<<grid, D * D / 32, 0, s>>>(set);
    else
        attn_rec_kernel<TI, D, false><<<grid, D * D / 32, 0, s>>>(set);
}

cudaError_t launch_attn_rec(const AttnSet &set, int nwalks, int D, int dtype, bool state_only, cudaStream_t s) {
    if (dtype == MGS_BF16)
        D == 64 ? rec_go<bf16, 64>(set, nwalks, state_only, s) : rec_go<bf16, 128>(set, nwalks, state_only, s);
    else
        D == 64 ? rec_go<float, 64>(set, nwalks, state_only, s) : rec_go<float, 128>(set, nwalks, state_only, s);
    return cudaGetLastError();
}

size_t attn_workspace_bytes(const mgs_attention_shape &sh, bool backward) {
    const Plan p = plan_of(sh, backward ? 3 : 1);
    size_t n = seg_bytes(p, sh.D) * (backward ? 3 : 1);
    n += 2 * split_bytes(sh, p, sh.Hk) + split_bytes(sh, p, sh.H) * (backward ? 2 : 1);
    if (backward) {
        const size_t rows = size_t(sh.B) * sh.T * sh.H;
        n += 2 * up256(rows * 4 * p.parts);                                                     // row products
        n += 2 * up256(size_t(p.lanes) * p.spans * sh.D * sh.D * 4);                  // S and R at span ends
        n += up256(size_t(p.lanes) * p.spans * 8);                                    // spans' sums of dg
        if (sh.Hk != sh.H) n += 2 * up256(rows * sh.D * 4);                           // dq, dk of each value head
    }
    return n;
}

cudaError_t launch_attn_fwd(const mgs_attention_shape &sh, const void *q, const void *k, const void *v,
                            const float *g, const float *S0, void *o, float *ST, void *ws, const DevCtl &ctl,
                            cudaStream_t s) {
    const Plan p = plan_of(sh, 1);
    Carve carve{static_cast<char *>(ws)};
    AttnSet set = set_of(sh, p, g, ctl);
    AttnWalk &w = set.w[0];
    Splitter split{sh, p, carve};
    w.q = split.take(q, sh.q_stride, sh.Hk, w.qs), w.k = split.take(k, sh.k_stride, sh.Hk, w.ks);
    w.v = split.take(v, sh.v_stride, sh.H, w.vs), w.out = o;
    const cudaError_t e = split.run(s);
    if (e != cudaSuccess) return e;
    dense(w.os, sh.T, sh.H, sh.D);
    w.qdiv = w.kdiv = int(sh.H / sh.Hk);
    w.s_in = S0, w.s_out = ST;
    w.o_scale = sh.scale;
    return run_walks(set, 1, sh, p, carve, s);
}

cudaError_t launch_attn_bwd(const mgs_attention_shape &sh, const void *q, const void *k, const void *v,
                            const float *g, const float *S0, const void *go, const float *gST, void *dq, void *dk,
                            void *dv, float *dg, float *dS0, void *ws, const DevCtl &ctl, cudaStream_t s) {
    const Plan p = plan_of(sh, 3);
    const int group = int(sh.H / sh.Hk);
    const size_t rows = size_t(sh.B) * sh.T * sh.H;
    Carve carve{static_cast<char *>(ws)};
    float *u = carve.take<float>(rows * 4 * p.parts), *wd = carve.take<float>(rows * 4 * p.parts);
    const size_t ck = size_t(p.lanes) * p.spans * sh.D * sh.D * 4;
    float *ckS = carve.take<float>(ck), *ckR = carve.take<float>(ck);
    float2 *part = carve.take<float2>(size_t(p.lanes) * p.spans * 8);
    float *dqf = nullptr, *dkf = nullptr;
    if (group > 1) dqf = carve.take<float>(rows * sh.D * 4), dkf = carve.take<float>(rows * sh.D * 4);
    AttnSet set = set_of(sh, p, g, ctl);
    set.kept = p.spans - (gST == nullptr ? 1 : 0);  // without a gradient of the last state R is zero there
    AttnWalk &a = set.w[0], &r = set.w[1], &c = set.w[2];
    Splitter split{sh, p, carve};
    int64_t qs[3], ks[3], vs[3], gs[3];
    const void *tq = split.take(q, sh.q_stride, sh.Hk, qs), *tk = split.take(k, sh.k_stride, sh.Hk, ks);
    const void *tv = split.take(v, sh.v_stride, sh.H, vs), *tg = split.take(go, sh.do_stride, sh.H, gs);
    cudaError_t e = split.run(s);
    if (e != cudaSuccess) return e;
    // dq = scale S do: the walk of (do, v, k) on S^T
    a.q = tg, a.k = tv, a.v = tk, a.x = q;
    copy3(a.qs, gs), copy3(a.ks, vs), copy3(a.vs, ks), copy3(a.xs, sh.q_stride);
    a.vdiv = a.xdiv = group;
    a.s_in = S0, a.s_in_t = 1, a.o_scale = sh.scale;
    a.row_dot = u, a.ckpt = set.kept > 0 ? ckS : nullptr;
    // dk = R v: the reverse walk of (v, do, q) on R^T
    r.q = tv, r.k = tg, r.v = tq, r.x = k;
    copy3(r.qs, vs), copy3(r.ks, gs), copy3(r.vs, qs), copy3(r.xs, sh.k_stride);
    r.vdiv = r.xdiv = group;
    r.s_in = gST, r.s_in_t = 1, r.kv_scale = sh.scale, r.rev = 1;
    r.row_dot = wd, r.ckpt = set.kept > 0 ? ckR : nullptr;
    // dv = R^T k: the reverse walk of (k, q, do) on R
    c.q = tk, c.k = tq, c.v = tg, c.out = dv;
    copy3(c.qs, ks), copy3(c.ks, qs), copy3(c.vs, gs);
    c.qdiv = c.kdiv = group;
    c.s_in = gST, c.s_out = dS0, c.kv_scale = sh.scale, c.rev = 1;
    dense(c.os, sh.T, sh.H, sh.D);
    // shared query/key heads: each value head's gradient in fp32, summed after
    dense(a.os, sh.T, sh.H, sh.D), dense(r.os, sh.T, sh.H, sh.D);
    a.out = group > 1 ? static_cast<void *>(dqf) : dq, a.out_f32 = group > 1;
    r.out = group > 1 ? static_cast<void *>(dkf) : dk, r.out_f32 = group > 1;
    if ((e = run_walks(set, 3, sh, p, carve, s)) != cudaSuccess) return e;
    if ((e = launch_next(attn_dg_kernel, unsigned(p.lanes * p.spans), 256, 0, s, p.mma, u, wd, p.parts,
                         ckS, ckR, sh.fixed_decay ? nullptr : dg, sh.fixed_decay ? part : nullptr, sh.T, sh.H, p.spans,
                         set.kept, p.span, sh.D * sh.D)) != cudaSuccess)
        return e;
    if (sh.fixed_decay) attn_dg_fixed_kernel<<<unsigned(sh.H), 256, 0, s>>>(part, dg, sh.B, sh.H, p.spans);
    if (group > 1) {
        const int64_t n4 = int64_t(rows) / group * sh.D / 4;
        const unsigned grid = unsigned(min64((n4 + 255) / 256, 152 * 8));
        for (int i = 0; i < 2; ++i) {
            const float *in = i ? dkf : dqf;
            void *out = i ? dk : dq;
            if (sh.dtype == MGS_BF16)
                attn_group_sum_kernel<<<grid, 256, 0, s>>>(in, static_cast<bf16 *>(out), n4, sh.D / 4, sh.Hk, group);
            else
                attn_group_sum_kernel<<<grid, 256, 0, s>>>(in, static_cast<float *>(out), n4, sh.D / 4, sh.Hk, group);
        }
    }
    return cudaGetLastError();
}

template <typename TI, int D>
static void step_go(const mgs_attention_shape &sh, const void *q, const void *k, const void *v, const float *g,
                    float *S, const int32_t *slots, int64_t nslots, void *o, cudaStream_t s) {
    attn_step_kernel<TI, D><<<unsigned(sh.B * sh.H * (D / 32)), 256, 0, s>>>(
        static_cast<const TI *>(q), static_cast<const TI *>(k), static_cast<const TI *>(v), g, S, slots,
        static_cast<TI *>(o), sh, nslots);
}

cudaError_t launch_attn_step(const mgs_attention_shape &sh, const void *q, const void *k, const void *v,
                             const float *g, float *S, const int32_t *slots, int64_t nslots, void *o,
                             cudaStream_t s) {
    if (sh.dtype == MGS_BF16)
        sh.D == 64 ? step_go<bf16, 64>(sh, q, k, v, g, S, slots, nslots, o, s)
                   : step_go<bf16, 128>(sh, q, k, v, g, S, slots, nslots, o, s);
    else
        sh.D == 64 ? step_go<float, 64>(sh, q, k, v, g, S, slots, nslots, o, s)
                   : step_go<float, 128>(sh, q, k, v, g, S, slots, nslots, o, s);
    return cudaGetLastError();
}

}  // namespace mgs
