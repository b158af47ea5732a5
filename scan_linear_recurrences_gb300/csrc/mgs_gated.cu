// The gated linear recurrence (minGRU) from its pre-activations.  Per channel, with
// z = sigmoid(gate) and c = value, or c = g(value) where g(v) = v + 1/2 for v >= 0,
// sigmoid(v) below,
//   h_t = (1 - z_t) h_{t-1} + z_t c_t.
// Backward, with a = 1 - z = sigmoid(-gate) and L_t = dL/dh_t = gh_t + a_{t+1} L_{t+1}:
//   dvalue = L z c',  dgate = L (c - h_{t-1}) z a,  dh0 = a_1 L_1.
//
// A run of steps acts on the state before it as s -> A s + H (A the product of its
// a, H its states from zero), and on the gradient behind it as f -> A f + R.  A
// block owns 64 channels of one sequence, each of its warps kSteps consecutive
// steps of a tile of kTile, a lane two channels: the inputs are read once and stay
// in registers, the warps exchange their maps through shared memory, and each runs
// its steps again from its own state.  With few channels a cluster of blocks takes
// tiles in turn, the blocks' maps pushed into each other's shared memory: one
// barrier of the cluster a round.
// The backward rebuilds h within a tile from the state that the forward kept before
// it (the carries), so that h is not read: five tensors pass, not six.
#include "mgs_cluster.cuh"
#include "mgs_lm.h"
#include "mgs_num.cuh"

namespace mgs {
namespace {

constexpr int kSteps = 8, kWarps = 8, kTile = kSteps * kWarps;
static_assert(kTile == MGS_GATED_SPAN, "a tile begins at a kept state");
constexpr int kMaxCluster = 16;

// Two channels in one register pair: sm_100 has fp32 sums and products of pairs
struct f2 {
    unsigned long long v;
};
__device__ __forceinline__ f2 pair(float x, float y) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 both(f2 p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p.v));
    return r;
}
__device__ __forceinline__ f2 operator+(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 operator*(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// e^-|x|.  bf16: the argument of the base-2 exponential is rounded (an error of |x|
// 2^-24); fp32: what the rounding left is made up for.
constexpr float kLog2e = 1.44269504f, kLog2eLow = 1.92596299e-8f, kLn2 = 0.693147181f;
template <typename T>
__device__ __forceinline__ float exp_minus(float x) {
    if constexpr (sizeof(T) == 2) return ex2_approx(-fabsf(x) * kLog2e);
    const float y = max_nan(-fabsf(x), -120.f);  // (zero from there on; NaN stays)
    const float t = y * kLog2e;
    const float low = fmaf(y, kLog2e, -t) + y * kLog2eLow;
    const float e = ex2_approx(t);
    return fmaf(e * kLn2, low, e);
}

// z, a = 1 - z and c of one step of two channels; z and a both to their own last
// digits.  Two sigmoids share one reciprocal, of the product of their denominators
// (both in 1..2).  Where z is zero in fp32 (a gate of -infinity, or of the type's
// lowest value) the step is masked: c is zero whatever the value.  A NaN in the
// value stays out of z and a, with which gradients pass.
template <typename T, bool POS>
__device__ __forceinline__ void gates(float2 k, float2 v, f2 &z, f2 &a, f2 &c) {
    const f2 one = pair(1.f, 1.f);
    const f2 e = pair(exp_minus<T>(k.x), exp_minus<T>(k.y));
    const f2 d = e + one;
    const float2 dd = both(d);
    f2 r, fs;
    if constexpr (POS) {
        const f2 f = pair(exp_minus<T>(v.x), exp_minus<T>(v.y));
        float2 g = both(f + one);
        g.x = fminf(g.x, 2.f), g.y = fminf(g.y, 2.f);  // (2 for NaN)
        const f2 gg = pair(g.x, g.y);
        const float2 p = both(d * gg);
        const f2 q = pair(rcp_approx(p.x), rcp_approx(p.y));
        r = q * gg;
        fs = f * (q * d);
    } else {
        r = pair(rcp_approx(dd.x), rcp_approx(dd.y));
    }
    // the smaller of z and a; the larger is 1 less it, rounded once: 1 where z is nothing beside it, so that a state
    // behind many such steps does not drift
    const f2 low = e * r;
    const float2 lo = both(low), hi = both(fma2(low, pair(-1.f, -1.f), one));
    const float2 zz = make_float2(k.x >= 0.f ? hi.x : lo.x, k.y >= 0.f ? hi.y : lo.y);
    z = pair(zz.x, zz.y);
    a = pair(k.x >= 0.f ? lo.x : hi.x, k.y >= 0.f ? lo.y : hi.y);
    float2 cc = v;
    if constexpr (POS) {
        const float2 up = both(pair(v.x, v.y) + pair(0.5f, 0.5f)), down = both(fs);
        // below zero less than 1/2, so that c tells the side (sigmoid of -1e-9 rounds to 1/2)
        cc.x = v.x < 0.f ? fminf(down.x, 0x1.fffffep-2f) : up.x;
        cc.y = v.y < 0.f ? fminf(down.y, 0x1.fffffep-2f) : up.y;
    }
    c = pair(zz.x == 0.f ? 0.f : cc.x, zz.y == 0.f ? 0.f : cc.y);
}

// Two channels of a step as they lie in memory: neighbours (VEC: one load), or 32
// apart (any alignment; `ok` has a bit for each).
template <typename T, bool VEC>
struct Two;
template <bool VEC>
struct Two<bf16, VEC> {
    uint32_t u;
    __device__ __forceinline__ void load(const bf16 *p, int ok) {
        if (VEC) {
            u = ok ? __ldcs(reinterpret_cast<const uint32_t *>(p)) : 0u;
        } else {
            const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
            u = (ok & 1 ? uint32_t(q[0]) : 0u) | (ok & 2 ? uint32_t(q[32]) << 16 : 0u);
        }
    }
    __device__ __forceinline__ float2 get() const { return make_float2(bf_lo(u), bf_hi(u)); }
    static __device__ __forceinline__ void store(bf16 *p, float2 v, int ok) {
        const uint32_t u = pack_bf16(v.x, v.y);
        if (VEC) {
            if (ok) __stcs(reinterpret_cast<uint32_t *>(p), u);
        } else {
            if (ok & 1) reinterpret_cast<uint16_t *>(p)[0] = uint16_t(u);
            if (ok & 2) reinterpret_cast<uint16_t *>(p)[32] = uint16_t(u >> 16);
        }
    }
};
template <bool VEC>
struct Two<float, VEC> {
    float2 u;
    __device__ __forceinline__ void load(const float *p, int ok) {
        if (VEC) u = ok ? __ldcs(reinterpret_cast<const float2 *>(p)) : make_float2(0.f, 0.f);
        else u = make_float2(ok & 1 ? p[0] : 0.f, ok & 2 ? p[32] : 0.f);
    }
    __device__ __forceinline__ float2 get() const { return u; }
    static __device__ __forceinline__ void store(float *p, float2 v, int ok) {
        if (VEC) {
            if (ok) __stcs(reinterpret_cast<float2 *>(p), v);
        } else {
            if (ok & 1) p[0] = v.x;
            if (ok & 2) p[32] = v.y;
        }
    }
};

struct Args {
    const void *gate, *value, *gh;
    void *h, *dgate, *dvalue;
    const float *in;    // forward: h0 (null: zeros); backward: the last state's gradient (null: zeros)
    float *out;         // forward: the last state; backward: dh0 (null: not wanted)
    float *carries;
    int64_t D, kb, kt, vb, vt, gb, gt;
    int T, tiles, strips, cluster;
};

// a lane's two channels of the block's 64, and which of them are there
template <bool VEC>
struct Lane {
    int64_t d;
    int ok;
    __device__ __forceinline__ Lane(int strip, int64_t D) {
        const int lane = threadIdx.x & 31;
        d = int64_t(strip) * 64 + (VEC ? 2 * lane : lane);
        ok = VEC ? (d < D ? 3 : 0) : (d < D ? 1 : 0) | (d + 32 < D ? 2 : 0);
    }
};

__device__ __forceinline__ void push16(void *slot, unsigned rank, float4 v) {
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dsmem_addr(slot, rank)), "f"(v.x), "f"(v.y),
                 "f"(v.z), "f"(v.w)
                 : "memory");
}

// One map of a lane's two channels
struct Map {
    f2 A, H;
    __device__ __forceinline__ float4 pack() const {
        const float2 a = both(A), h = both(H);
        return make_float4(a.x, a.y, h.x, h.y);
    }
    static __device__ __forceinline__ Map unpack(float4 m) { return {pair(m.x, m.y), pair(m.z, m.w)}; }
};

// The state that enters this warp's steps: `s` (the state before the round) through
// the maps before this warp's, and s through all of them for the next round.  REV:
// the maps act from the last warp, and the last block of the cluster, to the first.
template <bool CL, bool REV>
__device__ __forceinline__ f2 enter(const float4 (*maps)[32], float4 (*slots)[32], f2 &s, int warp, int lane,
                                    int cluster, unsigned rank) {
    f2 mine = s;
    if constexpr (!CL) {
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const int j = REV ? kWarps - 1 - i : i;
            if (j == warp) mine = s;
            const Map m = Map::unpack(maps[j][lane]);
            s = fma2(m.A, s, m.H);
        }
        return mine;
    }
    Map before{pair(1.f, 1.f), pair(0.f, 0.f)}, all = before;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        const int j = REV ? kWarps - 1 - i : i;
        if (j == warp) before = all;
        const Map m = Map::unpack(maps[j][lane]);
        all.H = fma2(m.A, all.H, m.H);
        all.A = m.A * all.A;
    }
    for (int r = warp; r < cluster; r += kWarps) push16(&slots[rank][lane], unsigned(r), all.pack());
    cluster_arrive();
    cluster_wait();
    for (int i = 0; i < cluster; ++i) {
        const int r = REV ? cluster - 1 - i : i;
        if (r == int(rank)) mine = s;
        const Map m = Map::unpack(slots[r][lane]);
        s = fma2(m.A, s, m.H);
    }
    return fma2(before.A, mine, before.H);
}

template <typename T, bool POS, bool VEC, bool CL>
__global__ void __launch_bounds__(kWarps * 32, 2) gated_fwd_kernel(const __grid_constant__ Args g) {
    __shared__ float4 maps[2][kWarps][32];
    __shared__ float4 slots[CL ? 2 : 1][CL ? kMaxCluster : 1][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cluster = CL ? g.cluster : 1;
    const unsigned rank = CL ? cluster_rank() : 0;
    const int strip = int(blockIdx.x / cluster % g.strips);
    const int64_t b = int64_t(blockIdx.x / cluster / g.strips);
    const Lane<VEC> at(strip, g.D);
    const T *gate = (const T *)g.gate + b * g.kb + at.d, *value = (const T *)g.value + b * g.vb + at.d;
    T *h = (T *)g.h + b * g.T * g.D + at.d;
    f2 s = pair(0.f, 0.f);
    if (g.in) {
        Two<float, VEC> x;
        x.load(g.in + b * g.D + at.d, at.ok);
        s = pair(x.u.x, x.u.y);
    }
    Two<T, VEC> rk[kSteps], rv[kSteps];
    auto fetch = [&](int tile) {
        const int t0 = tile * kTile + warp * kSteps;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int ok = t0 + i < g.T ? at.ok : 0;
            rk[i].load(gate + int64_t(t0 + i) * g.kt, ok);
            rv[i].load(value + int64_t(t0 + i) * g.vt, ok);
        }
    };
    fetch(int(rank));
    int turn = 0;
    for (int first = 0; first < g.tiles; first += cluster, turn ^= 1) {
        const int tile = first + int(rank), t0 = tile * kTile + warp * kSteps;
        f2 a[kSteps], c[kSteps];
        Map m{pair(1.f, 1.f), pair(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            f2 z;
            gates<T, POS>(rk[i].get(), rv[i].get(), z, a[i], c[i]);
            c[i] = z * c[i];
            if (t0 + i >= g.T) a[i] = pair(1.f, 1.f), c[i] = pair(0.f, 0.f);  // no step
            m.H = fma2(a[i], m.H, c[i]);
            m.A = m.A * a[i];
        }
        if (tile + cluster < g.tiles) fetch(tile + cluster);
        maps[turn][warp][lane] = m.pack();
        __syncthreads();
        f2 x = enter<CL, false>(maps[turn], slots[CL ? turn : 0], s, warp, lane, cluster, rank);
        if (g.carries && warp == 0 && tile < g.tiles)
            Two<float, VEC>::store(g.carries + (b * g.tiles + tile) * g.D + at.d, both(x), at.ok);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            x = fma2(a[i], x, c[i]);
            Two<T, VEC>::store(h + int64_t(t0 + i) * g.D, both(x), t0 + i < g.T ? at.ok : 0);
        }
    }
    if (g.out && rank == 0 && warp == 0) Two<float, VEC>::store(g.out + b * g.D + at.d, both(s), at.ok);
}

template <typename T, bool POS, bool VEC, bool CL>
__global__ void __launch_bounds__(kWarps * 32, 2) gated_bwd_kernel(const __grid_constant__ Args g) {
    __shared__ float4 maps[2][kWarps][32], back[2][kWarps][32];
    __shared__ float4 slots[CL ? 2 : 1][CL ? kMaxCluster : 1][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cluster = CL ? g.cluster : 1;
    const unsigned rank = CL ? cluster_rank() : 0;
    const int strip = int(blockIdx.x / cluster % g.strips);
    const int64_t b = int64_t(blockIdx.x / cluster / g.strips);
    const Lane<VEC> at(strip, g.D);
    const T *gate = (const T *)g.gate + b * g.kb + at.d, *value = (const T *)g.value + b * g.vb + at.d,
            *gh = (const T *)g.gh + b * g.gb + at.d;
    T *dgate = (T *)g.dgate + b * g.T * g.D + at.d, *dvalue = (T *)g.dvalue + b * g.T * g.D + at.d;
    f2 flow = pair(0.f, 0.f);
    if (g.in) {
        Two<float, VEC> x;
        x.load(g.in + b * g.D + at.d, at.ok);
        flow = pair(x.u.x, x.u.y);
    }
    Two<T, VEC> rk[kSteps], rv[kSteps], rg[kSteps];
    Two<float, VEC> rc;
    auto fetch = [&](int tile) {
        const int t0 = tile * kTile + warp * kSteps;
        rc.load(g.carries + (b * g.tiles + tile) * g.D + at.d, tile < g.tiles ? at.ok : 0);
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const int ok = t0 + i < g.T ? at.ok : 0;
            rk[i].load(gate + int64_t(t0 + i) * g.kt, ok);
            rv[i].load(value + int64_t(t0 + i) * g.vt, ok);
            rg[i].load(gh + int64_t(t0 + i) * g.gt, ok);
        }
    };
    int first = (g.tiles - 1) / cluster * cluster, turn = 0;
    fetch(first + int(rank));
    for (; first >= 0; first -= cluster, turn ^= 1) {
        const int tile = first + int(rank), t0 = tile * kTile + warp * kSteps;
        f2 a[kSteps], z[kSteps], c[kSteps];
        Two<T, VEC> gr[kSteps];
        Map m{pair(1.f, 1.f), pair(0.f, 0.f)};
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            gates<T, POS>(rk[i].get(), rv[i].get(), z[i], a[i], c[i]);
            if (t0 + i >= g.T) a[i] = pair(1.f, 1.f), z[i] = c[i] = pair(0.f, 0.f);
            m.H = fma2(a[i], m.H, z[i] * c[i]);
            m.A = m.A * a[i];
            gr[i] = rg[i];
        }
        const f2 start = pair(rc.u.x, rc.u.y);
        if (first > 0) fetch(tile - cluster);
        Map n{m.A, pair(0.f, 0.f)};
#pragma unroll
        for (int i = kSteps - 1; i >= 0; --i) {
            const float2 x = gr[i].get();
            n.H = a[i] * (pair(x.x, x.y) + n.H);
        }
        maps[turn][warp][lane] = m.pack();
        back[turn][warp][lane] = n.pack();
        __syncthreads();
        f2 x = start;  // the state before this warp's steps
        for (int j = 0; j < warp; ++j) {
            const Map o = Map::unpack(maps[turn][j][lane]);
            x = fma2(o.A, x, o.H);
        }
        // z <- z c', c <- (c - h before) z a
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            const f2 d = fma2(x, pair(-1.f, -1.f), c[i]), w = z[i] * d;
            x = x + w;
            if constexpr (POS) {
                const float2 cc = both(c[i]), lo = both(fma2(c[i] * pair(-1.f, -1.f), c[i], c[i]));
                z[i] = z[i] * pair(cc.x < 0.5f ? lo.x : 1.f, cc.y < 0.5f ? lo.y : 1.f);
            }
            c[i] = a[i] * w;
        }
        f2 f = enter<CL, true>(back[turn], slots[CL ? turn : 0], flow, warp, lane, cluster, rank);
#pragma unroll
        for (int i = kSteps - 1; i >= 0; --i) {
            const float2 y = gr[i].get();
            const f2 lam = pair(y.x, y.y) + f;
            const int ok = t0 + i < g.T ? at.ok : 0;
            Two<T, VEC>::store(dvalue + int64_t(t0 + i) * g.D, both(lam * z[i]), ok);
            Two<T, VEC>::store(dgate + int64_t(t0 + i) * g.D, both(lam * c[i]), ok);
            f = a[i] * lam;
        }
    }
    if (g.out && rank == 0 && warp == 0) Two<float, VEC>::store(g.out + b * g.D + at.d, both(flow), at.ok);
}

template <typename T, bool POS, bool VEC>
__global__ void __launch_bounds__(128)
    gated_step_kernel(const T *__restrict__ gate, const T *__restrict__ value, float *__restrict__ state,
                      const int32_t *__restrict__ slots, int64_t nslots, T *__restrict__ h, int64_t B, int64_t D,
                      int strips, int64_t kb, int64_t vb) {
    const int64_t i = int64_t(blockIdx.x) * 4 + threadIdx.x / 32, b = i / strips;
    if (b >= B) return;
    const Lane<VEC> at(int(i % strips), D);
    const int64_t slot = slots ? slots[b] : b;
    Two<T, VEC> k, v;
    k.load(gate + b * kb + at.d, at.ok);
    v.load(value + b * vb + at.d, at.ok);
    float2 x = make_float2(0.f, 0.f);
    if (slot >= 0 && slot < nslots) {
        Two<float, VEC> s;
        s.load(state + slot * D + at.d, at.ok);
        f2 z, a, c;
        gates<T, POS>(k.get(), v.get(), z, a, c);
        x = both(fma2(a, pair(s.u.x, s.u.y), z * c));
        Two<float, VEC>::store(state + slot * D + at.d, x, at.ok);
    }
    Two<T, VEC>::store(h + b * D + at.d, x, at.ok);
}

// channels in pairs: every row of every tensor starts at a multiple of two elements
bool pairs(const Args &g, int es) {
    auto ok = [&](const void *p, int size) { return reinterpret_cast<uintptr_t>(p) % unsigned(2 * size) == 0; };
    return ((g.D | g.kb | g.kt | g.vb | g.vt | g.gb | g.gt) & 1) == 0 && ok(g.gate, es) && ok(g.value, es) &&
           ok(g.gh, es) && ok(g.h, es) && ok(g.dgate, es) && ok(g.dvalue, es) && ok(g.in, 4) && ok(g.out, 4) &&
           ok(g.carries, 4);
}

// Blocks of a cluster: enough for two blocks an SM, as far as there are tiles
int cluster_of(int64_t lanes, int tiles) {
    int c = 1;
    while (c < kMaxCluster && lanes * c < 304 && c < tiles) c *= 2;
    return c;
}

template <typename F, typename C>
cudaError_t run(F *plain, C *clustered, Args &g, int64_t lanes, cudaStream_t s) {
    g.cluster = cluster_of(lanes, g.tiles);
    if (g.cluster > 1) return launch_cluster(clustered, lanes * g.cluster, kWarps * 32, 0, g.cluster, s, g);
    plain<<<unsigned(lanes), kWarps * 32, 0, s>>>(g);
    return cudaGetLastError();
}

Args args_of(const mgs_gated_shape &sh) {
    Args g = {};
    g.D = sh.D, g.T = int(sh.T), g.tiles = int((sh.T + kTile - 1) / kTile), g.strips = int((sh.D + 63) / 64);
    g.kb = sh.gate_stride[0], g.kt = sh.gate_stride[1], g.vb = sh.value_stride[0], g.vt = sh.value_stride[1];
    return g;
}
template <typename T, bool POS>
cudaError_t fwd_go(const mgs_gated_shape &sh, Args &g, cudaStream_t s) {
    const int64_t lanes = sh.B * g.strips;
    return pairs(g, sizeof(T)) ? run(gated_fwd_kernel<T, POS, true, false>, gated_fwd_kernel<T, POS, true, true>, g, lanes, s)
                               : run(gated_fwd_kernel<T, POS, false, false>, gated_fwd_kernel<T, POS, false, true>, g, lanes, s);
}
template <typename T, bool POS>
cudaError_t bwd_go(const mgs_gated_shape &sh, Args &g, cudaStream_t s) {
    const int64_t lanes = sh.B * g.strips;
    return pairs(g, sizeof(T)) ? run(gated_bwd_kernel<T, POS, true, false>, gated_bwd_kernel<T, POS, true, true>, g, lanes, s)
                               : run(gated_bwd_kernel<T, POS, false, false>, gated_bwd_kernel<T, POS, false, true>, g, lanes, s);
}
template <typename T, bool POS>
cudaError_t step_go(const mgs_gated_shape &sh, Args &g, float *state, const int32_t *slots, int64_t nslots,
                    cudaStream_t s) {
    g.kt = g.vt = 0;
    g.out = state;
    auto *fn = pairs(g, sizeof(T)) ? gated_step_kernel<T, POS, true> : gated_step_kernel<T, POS, false>;
    fn<<<unsigned((sh.B * g.strips + 3) / 4), 128, 0, s>>>((const T *)g.gate, (const T *)g.value, state, slots, nslots,
                                                          (T *)g.h, sh.B, sh.D, g.strips, g.kb, g.vb);
    return cudaGetLastError();
}

}  // namespace

#define MGS_BY_TYPE(go, ...)                                                                              \
    (sh.dtype == MGS_BF16 ? (sh.positive ? go<bf16, true>(__VA_ARGS__) : go<bf16, false>(__VA_ARGS__))    \
                          : (sh.positive ? go<float, true>(__VA_ARGS__) : go<float, false>(__VA_ARGS__)))

cudaError_t launch_gated_fwd(const mgs_gated_shape &sh, const void *gate, const void *value, const float *h0, void *h,
                             float *hT, float *carries, cudaStream_t s) {
    Args g = args_of(sh);
    g.gate = gate, g.value = value, g.in = h0, g.h = h, g.out = hT, g.carries = carries;
    return MGS_BY_TYPE(fwd_go, sh, g, s);
}
cudaError_t launch_gated_bwd(const mgs_gated_shape &sh, const void *gate, const void *value, const float *carries,
                             const void *gh, const float *ghT, void *dgate, void *dvalue, float *dh0, cudaStream_t s) {
    Args g = args_of(sh);
    g.gate = gate, g.value = value, g.carries = const_cast<float *>(carries), g.gh = gh, g.in = ghT;
    g.dgate = dgate, g.dvalue = dvalue, g.out = dh0, g.gb = sh.gh_stride[0], g.gt = sh.gh_stride[1];
    return MGS_BY_TYPE(bwd_go, sh, g, s);
}
cudaError_t launch_gated_step(const mgs_gated_shape &sh, const void *gate, const void *value, float *state,
                              const int32_t *slots, int64_t nslots, void *h, cudaStream_t s) {
    Args g = args_of(sh);
    g.gate = gate, g.value = value, g.h = h;
    return MGS_BY_TYPE(step_go, sh, g, state, slots, nslots, s);
}
#undef MGS_BY_TYPE

}  // namespace mgs
