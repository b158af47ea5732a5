// The gated linear recurrence (minGRU) from its pre-activations.  Per channel, with
// z = sigmoid(gate) and c = value, or c = g(value) where g(v) = v + 1/2 for v >= 0,
// sigmoid(v) below,
//   h_t = (1 - z_t) h_{t-1} + z_t c_t.
// Backward, with a = 1 - z = sigmoid(-gate) and L_t = dL/dh_t = gh_t + a_{t+1} L_{t+1}:
//   dvalue = L z c',  dgate = L (c - h_{t-1}) z a,  dh0 = a_1 L_1.
//
// A run of steps acts on the state before it as s -> A s + H (A the product of its
// a, H its states from zero), and on the gradient behind it as f -> A f + R.  A
// block owns 64 channels of one sequence, each of its warps consecutive steps of a
// tile of 64, a lane two channels.  A warp copies its part of the next tile to
// shared memory while it works on this one's, keeps what it computes in registers,
// exchanges its map with the other warps' and runs its steps again from its own
// state: the inputs are read once.  With few channels a cluster of blocks takes
// tiles in turn, their maps pushed into each other's shared memory (mgs_rounds.h).
// The backward rebuilds h within a tile from the state that the forward kept before
// it (the carries), so that h is not read: five tensors pass, not six.
//
// fp32 is bound by memory: 16 x 4096 x 1024 forward 127 us (6.3 TB/s), backward 226
// (5.9).  bf16, with half the bytes and as much to compute, by latency at 16 warps an SM:
// 8 x 4096 x 2048 forward 83 us (4.9, with the carries), backward 148 (4.5), in which 28
// and about 50 instructions a step and channel fill two thirds of the issue slots; and by
// the spread of the blocks, two on some SMs and one on others: 4096 steps take 49 and 87 us
// with 152 blocks, 83 and 149 with 256, 84 and 151 (5.7 and 5.3 TB/s) with 304.  Few
// channels are bound by the exchange: 1 x 16384 x 2048 in bf16, clusters of 16, 60 us (3.3),
// in fp32, clusters of 8, 94 (4.3).
#include <type_traits>

#include "mgs_cluster.cuh"
#include "mgs_launch.h"
#include "mgs_lm.h"
#include "mgs_num.cuh"
#include "mgs_rounds.h"

namespace mgs {
namespace {

constexpr int kTile = MGS_GATED_SPAN;  // a tile begins at a kept state
constexpr int kMaxCluster = 16;

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

// z, a = 1 - z, c and z c' (BWD) of one step of two channels; z and a both to
// their own last digits.  Two sigmoids share one reciprocal, of the product of their
// denominators (both in 1..2).  BWD: a NaN in the value stays out of z and a, with
// which gradients pass to the steps before (its own slope and the states behind it are
// NaN).
template <typename T, bool POS, bool BWD>
__device__ __forceinline__ void gates(float2 k, float2 v, f2 &z, f2 &a, f2 &c, f2 &zs) {
    const f2 one = pair(1.f, 1.f);
    const f2 e = pair(exp_minus<T>(k.x), exp_minus<T>(k.y));
    const f2 d = e + one;
    f2 r, s, fs;
    if constexpr (POS) {
        const f2 f = pair(exp_minus<T>(v.x), exp_minus<T>(v.y));
        f2 g = f + one;
        if constexpr (BWD) {
            const float2 gg = both(g);
            g = pair(fminf(gg.x, 2.f), fminf(gg.y, 2.f));  // (2 for NaN)
        }
        const float2 p = both(d * g);
        const f2 q = pair(rcp_approx(p.x), rcp_approx(p.y));
        r = q * g;
        s = q * d;
        fs = f * s;
    } else {
        const float2 p = both(d);
        r = pair(rcp_approx(p.x), rcp_approx(p.y));
    }
    // the smaller of z and a; the larger is 1 less it, rounded once: 1 where z is nothing beside it, so that a state
    // behind many such steps does not drift
    const f2 low = e * r;
    const float2 lo = both(low), hi = both(fma2(low, pair(-1.f, -1.f), one));
    const bool kx = k.x >= 0.f, ky = k.y >= 0.f;
    z = pair(kx ? hi.x : lo.x, ky ? hi.y : lo.y);
    a = pair(kx ? lo.x : hi.x, ky ? lo.y : hi.y);
    c = pair(v.x, v.y);
    zs = z;
    if constexpr (POS) {
        const bool vx = !(v.x >= 0.f), vy = !(v.y >= 0.f);  // (a NaN has the slope of NaN)
        const float2 up = both(c + pair(0.5f, 0.5f)), down = both(fs);
        c = pair(vx ? down.x : up.x, vy ? down.y : up.y);
        if constexpr (BWD) {
            const float2 slope = both(fs * s);
            zs = z * pair(vx ? slope.x : 1.f, vy ? slope.y : 1.f);
        }
    }
}

// Two channels of a step: neighbours (VEC), or 32 apart (any alignment; `ok` has a
// bit for each).
constexpr float kMasked = -88.f;  // z is zero in fp32: the step is masked, whatever its value
template <typename T, bool VEC>
struct Two;
template <bool VEC>
struct Two<bf16, VEC> {
    uint32_t u;
    __device__ __forceinline__ void load(const bf16 *p, int ok) {
        if (VEC) {
            u = ok ? *reinterpret_cast<const uint32_t *>(p) : 0u;
        } else {
            const uint16_t *q = reinterpret_cast<const uint16_t *>(p);
            u = (ok & 1 ? uint32_t(q[0]) : 0u) | (ok & 2 ? uint32_t(q[32]) << 16 : 0u);
        }
    }
    __device__ __forceinline__ float2 get() const { return make_float2(bf_lo(u), bf_hi(u)); }
    // the value, zero where its gate masks it
    __device__ __forceinline__ float2 get_unmasked(const Two &gate) const {
        const __nv_bfloat162 k = *reinterpret_cast<const __nv_bfloat162 *>(&gate.u);
        const uint32_t x = u & __hgeu2_mask(k, __float2bfloat162_rn(kMasked));  // (NaN: not masked)
        return make_float2(bf_lo(x), bf_hi(x));
    }
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
        if (VEC) u = ok ? *reinterpret_cast<const float2 *>(p) : make_float2(0.f, 0.f);
        else u = make_float2(ok & 1 ? p[0] : 0.f, ok & 2 ? p[32] : 0.f);
    }
    __device__ __forceinline__ float2 get() const { return u; }
    __device__ __forceinline__ float2 get_unmasked(const Two &gate) const {
        return make_float2(gate.u.x < kMasked ? 0.f : u.x, gate.u.y < kMasked ? 0.f : u.y);
    }
    static __device__ __forceinline__ void store(float *p, float2 v, int ok) {
        if (VEC) {
            if (ok) __stcs(reinterpret_cast<float2 *>(p), v);
        } else {
            if (ok & 1) p[0] = v.x;
            if (ok & 2) p[32] = v.y;
        }
    }
};

// How a warp's steps come to shared memory: copies of 16 bytes (rows that start at
// such multiples), of 4 bytes, or element by element (bf16 that starts anywhere).
enum Copy { kCopy16, kCopy4, kCopyAny };
__device__ __forceinline__ void copy16(void *dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(void *dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(ok ? 4 : 0) : "memory");
}
__device__ __forceinline__ void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Rows 0 .. n - 1 of L of 64 channels (zeros behind them and past the `left` that are
// there), `stride` apart, from `src` (any address of the tensor where n <= 0) to a
// warp's [L][64].
template <typename T, int L, Copy HOW>
__device__ __forceinline__ void copy_rows(T *dst, const T *src, int64_t stride, int n, int64_t left) {
    const int lane = threadIdx.x & 31;
    if constexpr (HOW == kCopy16) {
        constexpr int V = 16 / int(sizeof(T)), PER = 64 / V, ROWS = 32 / PER;  // lanes a row, rows at once
        const int row = lane / PER, col = lane % PER * V;
        const bool in = col < left;
        const T *p = src + row * stride + col;
        if (n >= L && left >= 64) {
#pragma unroll
            for (int i = 0; i < L / ROWS; ++i) {
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst + (i * ROWS + row) * 64 + col)), "l"(p) : "memory");
                p += ROWS * stride;
            }
            return;
        }
#pragma unroll
        for (int i = 0; i < L / ROWS; ++i) {
            const bool ok = in && i * ROWS + row < n;
            copy16(dst + (i * ROWS + row) * 64 + col, ok ? p + i * ROWS * stride : src, ok);
        }
    } else if constexpr (HOW == kCopy4) {
        constexpr int V = 4 / int(sizeof(T));
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int j = 0; j < 2 / V; ++j) {
                const int col = lane * V + 32 * j;
                const bool ok = col < left && i < n;
                copy4(dst + i * 64 + col, ok ? src + i * stride + col : src, ok);
            }
    } else {
        T x[L][2];
#pragma unroll
        for (int i = 0; i < L; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                x[i][j] = lane + 32 * j < left && i < n ? src[i * stride + lane + 32 * j] : from_f<T>(0.f);
#pragma unroll
        for (int i = 0; i < L; ++i) dst[i * 64 + lane] = x[i][0], dst[i * 64 + lane + 32] = x[i][1];
    }
}

struct Args {
    const void *gate, *value, *gh;
    void *h, *dgate, *dvalue;
    const float *in;    // forward: h0 (null: zeros); backward: the last state's gradient (null: zeros)
    float *out;         // forward: the last state; backward: dh0 (null: not wanted)
    float *carries;
    int64_t D, kb, kt, vb, vt, gb, gt;
    int T, tiles, strips, cluster;
    DevCtl ctl;
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

// One map of a lane's two channels
struct Map {
    f2 A, H;
    __device__ __forceinline__ float4 pack() const {
        const float2 a = both(A), h = both(H);
        return make_float4(a.x, a.y, h.x, h.y);
    }
    static __device__ __forceinline__ Map unpack(float4 m) { return {pair(m.x, m.y), pair(m.z, m.w)}; }
};

// 16 bytes into shared memory of the cluster's CTA `rank`, counted by its barrier
__device__ __forceinline__ void push16(void *slot, uint64_t *bar, unsigned rank, float4 v) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                     dsmem_addr(slot, rank)),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(dsmem_addr(bar, rank))
                 : "memory");
}

// The maps of a tile's warps, and of a round's blocks (CL): two of each, in turn.
template <int W, bool CL>
struct Exchange {
    float4 maps[2][W][32];
    float4 slots[2][kMaxCluster][32];
    alignas(16) uint64_t bar[2];
    unsigned gave_up[2];  // up to a round of that turn a wait has
    unsigned pushed;      // the rounds in which this block has pushed its map
    unsigned told;        // some block's wait has given up
};
// Without a cluster: what the last warp leaves to the next tile.  (Two blocks of the
// backward in fp32 fill an SM's shared memory to the last KB.)
template <int W>
struct Exchange<W, false> {
    float4 maps[2][W][32];
    unsigned long long pass[2][32];
};

// The state that enters this warp's steps: what the last warp had after its own in the
// tile before, through the maps of this tile's warps before this one (REV: the maps act
// from the last warp to the first).
template <bool REV, int W>
__device__ __forceinline__ f2 enter(const Exchange<W, false> &ex, int turn, int warp, int lane) {
    f2 s{ex.pass[turn ^ 1][lane]};
#pragma unroll
    for (int i = 0; i < W - 1; ++i) {
        const int j = REV ? W - 1 - i : i;
        if (REV ? j > warp : j < warp) {
            const Map m = Map::unpack(ex.maps[turn][j][lane]);
            s = fma2(m.A, s, m.H);
        }
    }
    return s;
}
// The steps of exchange_round and leave_rounds, by a thread
template <int W>
struct Ops {
    Exchange<W, true> &ex;
    int warp, lane, cluster;
    unsigned self;
    const DevCtl &ctl;
    float4 map;  // the block's
    __device__ __forceinline__ bool gave_up(int turn) const { return *const_cast<volatile unsigned *>(&ex.gave_up[turn]) != 0; }
    __device__ __forceinline__ void stay_out(int turn) const { *const_cast<volatile unsigned *>(&ex.gave_up[turn]) = 1u; }
    __device__ __forceinline__ void give_up(int turn) const {
        stay_out(turn);
        record_error(ctl, ERR_MBAR_TIMEOUT);
    }
    __device__ __forceinline__ void push(int turn) const {
        for (int r = warp; r < cluster; r += W) push16(&ex.slots[turn][self][lane], &ex.bar[turn], unsigned(r), map);
    }
    __device__ __forceinline__ void count_and_arm(int turn) const {
        if (warp != 0 || lane != 0) return;
        mbar_arrive_expect_tx(&ex.bar[turn], unsigned(cluster) * 512u);
        atomicAdd(&ex.pushed, 1u);
    }
    __device__ __forceinline__ bool wait(int turn, int phase) const {
        return mbar_wait_bounded(&ex.bar[turn], unsigned(phase), ctl.timeout_ns);
    }
    __device__ __forceinline__ void block_barrier() const { __syncthreads(); }
    __device__ __forceinline__ void cluster_barrier() const { cluster_arrive(), cluster_wait(); }
    __device__ __forceinline__ void tell_all() const {
        if (int(threadIdx.x) < cluster) st_dsmem_u32(&ex.told, threadIdx.x, 1u);
    }
    __device__ __forceinline__ bool told() const { return *const_cast<volatile unsigned *>(&ex.told) != 0; }
    __device__ __forceinline__ bool first_warp() const { return warp == 0; }
    __device__ __forceinline__ unsigned rank() const { return self; }
    __device__ __forceinline__ int pushed(unsigned r) const { return int(ld_dsmem_u32(&ex.pushed, r)); }
    __device__ __forceinline__ void stand_in(int r, int turn) const {
        push16(&ex.slots[turn][r][lane], &ex.bar[turn], self, make_float4(0.f, 0.f, 0.f, 0.f));
    }
    __device__ __forceinline__ void arm(int turn, int blocks) const {
        if (lane == 0) mbar_arrive_expect_tx(&ex.bar[turn], unsigned(blocks) * 512u);
        __syncwarp();
    }
    __device__ __forceinline__ void not_drained() const { record_error(ctl, ERR_DRAIN_TIMEOUT); }
};

// In a cluster: `s` (the state before the round, which every block keeps) through the
// maps of the blocks before this one and of the warps before this one, and s through
// all of them for the next round.  (Of no meaning where a wait gave up.)
template <bool REV, int W>
__device__ __forceinline__ f2 enter(Ops<W> op, int round, f2 &s) {
    const Exchange<W, true> &ex = op.ex;
    const int turn = round & 1;
    f2 mine = s;
    Map before{pair(1.f, 1.f), pair(0.f, 0.f)}, all = before;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        const int j = REV ? W - 1 - i : i;
        if (j == op.warp) before = all;
        const Map m = Map::unpack(ex.maps[turn][j][op.lane]);
        all.H = fma2(m.A, all.H, m.H);
        all.A = m.A * all.A;
    }
    op.map = all.pack();
    exchange_round(op, round);
    for (int i = 0; i < op.cluster; ++i) {
        const int r = REV ? op.cluster - 1 - i : i;
        if (r == int(op.self)) mine = s;
        const Map m = Map::unpack(ex.slots[turn][r][op.lane]);
        s = fma2(m.A, s, m.H);
    }
    return fma2(before.A, mine, before.H);
}

// all blocks of the cluster have their barriers before the first push
template <int W>
__device__ __forceinline__ void meet(Exchange<W, true> &ex) {
    if (threadIdx.x == 0) {
        mbar_init(&ex.bar[0], 1), mbar_init(&ex.bar[1], 1);
        ex.gave_up[0] = ex.gave_up[1] = ex.pushed = ex.told = 0u;
        fence_barrier_init();
    }
    __syncthreads();
    cluster_arrive();
    cluster_wait();
}

// The exchange by itself, between the blocks of one cluster, one of which may come late to a
// round: how many rounds each took part in, and how many messages it found wrong in them.
constexpr int kCheckBlocks = MGS_EXCHANGE_BLOCKS, kCheckRounds = MGS_EXCHANGE_ROUNDS, kCheckWarps = 4;
__global__ void __launch_bounds__(kCheckWarps * 32)
    exchange_check_kernel(int late_block, int late_round, uint64_t late_ns, int32_t *rounds, int32_t *wrong, DevCtl ctl) {
    __shared__ Exchange<kCheckWarps, true> ex;
    __shared__ int bad;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned rank = cluster_rank();
    Ops<kCheckWarps> op{ex, warp, lane, kCheckBlocks, rank, ctl, {}};
    if (threadIdx.x == 0) bad = 0;
    meet(ex);
    for (int n = 0; n < kCheckRounds; ++n) {
        if (int(rank) == late_block && n == late_round)
            for (const uint64_t t0 = global_ns(); global_ns() - t0 < late_ns;) __nanosleep(1000);
        __syncthreads();
        op.map = make_float4(float(n), float(rank), float(lane), 1.f);
        exchange_round(op, n);
        for (int r = 0; r < kCheckBlocks && !op.gave_up(n & 1); ++r) {
            const float4 m = ex.slots[n & 1][r][lane];
            if (m.x != float(n) || m.y != float(r) || m.z != float(lane) || m.w != 1.f) atomicAdd(&bad, 1);
        }
    }
    leave_rounds(op, kCheckBlocks);
    if (threadIdx.x != 0) return;
    rounds[rank] = int32_t(ex.pushed);
    wrong[rank] = atomicOr(ctl.err, 0u) & ERR_DRAIN_TIMEOUT ? -1 : bad;
}

// Warps of a forward's block and steps of its tile.  The maps cost the less the longer a
// warp's steps: 16 in bf16, by four warps in a cluster (more of them to a round; a prompt
// of 16384 x 2048 takes 60 us, 81 with eight), by eight without (8 x 4096 x 2048: 83 us,
// 86 with four); 8 in fp32, where, with twice the bytes, more warps pay.
template <typename T, bool CL>
constexpr int kFwdWarps = sizeof(T) == 2 && CL ? 4 : 8;
template <typename T, bool CL>
constexpr int kFwdTile = kFwdWarps<T, CL> * (sizeof(T) == 2 ? 16 : 8);
constexpr int kBwdWarps = 8;

template <typename T, bool POS, Copy HOW, bool CL>
__global__ void __launch_bounds__(kFwdWarps<T, CL> * 32, 512 / (kFwdWarps<T, CL> * 32))
    gated_fwd_kernel(const __grid_constant__ Args g) {
    constexpr int W = kFwdWarps<T, CL>, TILE = kFwdTile<T, CL>, L = TILE / W;
    constexpr bool VEC = HOW == kCopy16 || (HOW == kCopy4 && sizeof(T) == 2);
    using Ex = Exchange<W, CL>;
    extern __shared__ __align__(16) unsigned char smem[];
    Ex &ex = *reinterpret_cast<Ex *>(smem);
    T *ring = reinterpret_cast<T *>(smem + sizeof(Ex));  // [W][2 stages][2 tensors][L][64]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cluster = CL ? g.cluster : 1;
    const unsigned rank = CL ? cluster_rank() : 0;
    const int strip = int(blockIdx.x / cluster % g.strips);
    const int64_t b = int64_t(blockIdx.x / cluster / g.strips), left = g.D - int64_t(strip) * 64;
    const Lane<VEC> at(strip, g.D);
    const T *gate = (const T *)g.gate + b * g.kb + int64_t(strip) * 64,
            *value = (const T *)g.value + b * g.vb + int64_t(strip) * 64;
    T *h = (T *)g.h + b * g.T * g.D + at.d;
    T *mine = ring + warp * (2 * 2 * L * 64);
    auto op = [&] {
        if constexpr (CL) return Ops<W>{ex, warp, lane, cluster, rank, g.ctl, {}};
    };
    auto fetch = [&](int tile, int stage) {
        const int t0 = tile * TILE + warp * L, n = g.T - t0;
        T *to = mine + stage * (2 * L * 64);
        if (tile < g.tiles && n > 0) {
            copy_rows<T, L, HOW>(to, gate + t0 * g.kt, g.kt, n, left);
            copy_rows<T, L, HOW>(to + L * 64, value + t0 * g.vt, g.vt, n, left);
        }
        copies_close();
    };
    fetch(int(rank), 0);
    if constexpr (CL) meet(ex);
    f2 s = pair(0.f, 0.f);
    if (g.in) {
        Two<float, VEC> x;
        x.load(g.in + b * g.D + at.d, at.ok);
        s = pair(x.u.x, x.u.y);
    }
    if constexpr (!CL)
        if (warp == 0) ex.pass[1][lane] = s.v;
    for (int first = 0, round = 0; first < g.tiles; first += cluster, ++round) {
        const int turn = round & 1, tile = first + int(rank), t0 = tile * TILE + warp * L, n = g.T - t0;
        __syncwarp();  // the other stage has been read
        fetch(tile + cluster, turn ^ 1);
        copies_wait<1>();
        __syncwarp();
        const T *from = mine + turn * (2 * L * 64) + (VEC ? 2 * lane : lane);
        f2 a[L], c[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            Two<T, VEC> k, v;
            f2 z, zs;
            k.load(from + i * 64, 3), v.load(from + (L + i) * 64, 3);
            gates<T, POS, false>(k.get(), v.get_unmasked(k), z, a[i], c[i], zs);
            c[i] = z * c[i];
        }
        if (n < L) {  // no steps
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (i >= n) a[i] = pair(1.f, 1.f), c[i] = pair(0.f, 0.f);
        }
        Map m{a[0], c[0]};
#pragma unroll
        for (int i = 1; i < L; ++i) {
            m.H = fma2(a[i], m.H, c[i]);
            m.A = m.A * a[i];
        }
        ex.maps[turn][warp][lane] = m.pack();
        __syncthreads();
        f2 x;
        if constexpr (CL) x = enter<false>(op(), round, s);
        else x = enter<false>(ex, turn, warp, lane);
        if (g.carries && warp * L % kTile == 0 && n > 0)
            Two<float, VEC>::store(g.carries + (b * ((g.T - 1) / kTile + 1) + t0 / kTile) * g.D + at.d, both(x), at.ok);
        T *to = h + t0 * g.D;
        auto run = [&](auto all) {  // all: every step is there
#pragma unroll
            for (int i = 0; i < L; ++i) {
                x = fma2(a[i], x, c[i]);
                Two<T, VEC>::store(to, both(x), all.value || i < n ? at.ok : 0);
                to += g.D;
            }
        };
        if (n >= L) run(std::true_type());
        else run(std::false_type());
        if constexpr (!CL) {
            s = x;
            if (warp == W - 1) ex.pass[turn][lane] = x.v;
        }
    }
    // (steps behind the last one leave the state as it is)
    if (g.out && rank == 0 && warp == (CL ? 0 : W - 1)) Two<float, VEC>::store(g.out + b * g.D + at.d, both(s), at.ok);
    if constexpr (CL) leave_rounds(op(), cluster);
}

template <typename T, bool POS, Copy HOW, bool CL>
__global__ void __launch_bounds__(kBwdWarps * 32, 2) gated_bwd_kernel(const __grid_constant__ Args g) {
    constexpr int W = kBwdWarps, L = kTile / W;
    constexpr bool VEC = HOW == kCopy16 || (HOW == kCopy4 && sizeof(T) == 2);
    using Ex = Exchange<W, CL>;
    extern __shared__ __align__(16) unsigned char smem[];
    Ex &ex = *reinterpret_cast<Ex *>(smem);
    float4(*maps)[W][32] = reinterpret_cast<float4(*)[W][32]>(smem + sizeof(Ex));  // the states' maps [2][W][32]
    T *ring = reinterpret_cast<T *>(smem + sizeof(Ex) + sizeof(float4) * 2 * W * 32);  // [W][2 stages][3 tensors][L][64]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, cluster = CL ? g.cluster : 1;
    const unsigned rank = CL ? cluster_rank() : 0;
    const int strip = int(blockIdx.x / cluster % g.strips);
    const int64_t b = int64_t(blockIdx.x / cluster / g.strips), left = g.D - int64_t(strip) * 64;
    const Lane<VEC> at(strip, g.D);
    const T *gate = (const T *)g.gate + b * g.kb + int64_t(strip) * 64,
            *value = (const T *)g.value + b * g.vb + int64_t(strip) * 64,
            *gh = (const T *)g.gh + b * g.gb + int64_t(strip) * 64;
    T *dgate = (T *)g.dgate + b * g.T * g.D + at.d, *dvalue = (T *)g.dvalue + b * g.T * g.D + at.d;
    T *mine = ring + warp * (2 * 3 * L * 64);
    auto op = [&] {
        if constexpr (CL) return Ops<W>{ex, warp, lane, cluster, rank, g.ctl, {}};
    };
    Two<float, VEC> next;  // the state before the next tile
    auto fetch = [&](int tile, int stage) {
        const int t0 = tile * kTile + warp * L, n = g.T - t0;
        T *to = mine + stage * (3 * L * 64);
        const bool there = tile >= 0 && tile < g.tiles;
        next.load(g.carries + (b * g.tiles + tile) * g.D + at.d, there ? at.ok : 0);
        if (there && n > 0) {
            copy_rows<T, L, HOW>(to, gate + t0 * g.kt, g.kt, n, left);
            copy_rows<T, L, HOW>(to + L * 64, value + t0 * g.vt, g.vt, n, left);
        }
        if (tile >= 0) copy_rows<T, L, HOW>(to + 2 * L * 64, gh + (n > 0 ? t0 * g.gt : 0), g.gt, n, left);  // (zeros where no step is)
        copies_close();
    };
    int first = (g.tiles - 1) / cluster * cluster;
    fetch(first + int(rank), 0);
    if constexpr (CL) meet(ex);
    f2 flow = pair(0.f, 0.f);
    if (g.in) {
        Two<float, VEC> x;
        x.load(g.in + b * g.D + at.d, at.ok);
        flow = pair(x.u.x, x.u.y);
    }
    if constexpr (!CL)
        if (warp == 0) ex.pass[1][lane] = flow.v;
    for (int round = 0, turn = 0; first >= 0; first -= cluster, ++round, turn ^= 1) {
        const int tile = first + int(rank), t0 = tile * kTile + warp * L, n = g.T - t0;
        f2 x = pair(next.u.x, next.u.y);
        __syncwarp();  // the other stage has been read
        fetch(tile - cluster, turn ^ 1);
        copies_wait<1>();
        __syncwarp();
        const T *from = mine + turn * (3 * L * 64) + (VEC ? 2 * lane : lane);
        f2 a[L], z[L], c[L], zs[L];
#pragma unroll
        for (int i = 0; i < L; ++i) {
            Two<T, VEC> k, v;
            k.load(from + i * 64, 3), v.load(from + (L + i) * 64, 3);
            gates<T, POS, true>(k.get(), v.get_unmasked(k), z[i], a[i], c[i], zs[i]);
        }
        if (n < L) {  // no steps
#pragma unroll
            for (int i = 0; i < L; ++i)
                if (i >= n) a[i] = pair(1.f, 1.f), z[i] = c[i] = zs[i] = pair(0.f, 0.f);
        }
        auto gradient = [&](int i) {
            Two<T, VEC> y;
            y.load(from + (2 * L + i) * 64, 3);
            const float2 u = y.get();
            return pair(u.x, u.y);
        };
        Map m{a[0], z[0] * c[0]}, r{a[0], pair(0.f, 0.f)};
#pragma unroll
        for (int i = 1; i < L; ++i) {
            m.H = fma2(a[i], m.H, z[i] * c[i]);
            m.A = m.A * a[i];
        }
        r.A = m.A;
#pragma unroll
        for (int i = L - 1; i >= 0; --i) r.H = a[i] * (gradient(i) + r.H);
        maps[turn][warp][lane] = m.pack();
        ex.maps[turn][warp][lane] = r.pack();
        __syncthreads();
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            if (j < warp) {
                const Map o = Map::unpack(maps[turn][j][lane]);
                x = fma2(o.A, x, o.H);
            }
        }
#pragma unroll
        for (int i = 0; i < L; ++i) {  // c <- z a (c - h before); x as the forward has it (x + z (c - x) keeps the
            const f2 w = z[i] * fma2(x, pair(-1.f, -1.f), c[i]);  // rounding of a large x where a is nothing)
            x = fma2(a[i], x, z[i] * c[i]);
            c[i] = a[i] * w;
        }
        f2 f;
        if constexpr (CL) f = enter<true>(op(), round, flow);
        else f = enter<true>(ex, turn, warp, lane);
        T *to_k = dgate + (t0 + L - 1) * g.D, *to_v = dvalue + (t0 + L - 1) * g.D;
        auto run = [&](auto all) {  // all: every step is there
#pragma unroll
            for (int i = L - 1; i >= 0; --i) {
                const f2 lam = gradient(i) + f;
                const int ok = all.value || i < n ? at.ok : 0;
                Two<T, VEC>::store(to_v, both(lam * zs[i]), ok);
                Two<T, VEC>::store(to_k, both(lam * c[i]), ok);
                f = a[i] * lam;
                to_v -= g.D, to_k -= g.D;
            }
        };
        if (n >= L) run(std::true_type());
        else run(std::false_type());
        if constexpr (!CL) {
            flow = f;
            if (warp == 0) ex.pass[turn][lane] = f.v;
        }
    }
    if (g.out && rank == 0 && warp == 0) Two<float, VEC>::store(g.out + b * g.D + at.d, both(flow), at.ok);
    if constexpr (CL) leave_rounds(op(), cluster);
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
        f2 z, a, c, zs;
        gates<T, POS, false>(k.get(), v.get_unmasked(k), z, a, c, zs);
        x = both(fma2(a, pair(s.u.x, s.u.y), z * c));
        Two<float, VEC>::store(state + slot * D + at.d, x, at.ok);
    }
    Two<T, VEC>::store(h + b * D + at.d, x, at.ok);
}

// The widest copies that every row's start allows; channels in pairs (every output
// and state too) with 16 bytes, and in bf16 with 4
Copy copy_of(const Args &g, int es) {
    const void *in[] = {g.gate, g.value, g.gh}, *out[] = {g.h, g.dgate, g.dvalue}, *f32[] = {g.in, g.out, g.carries};
    const uint64_t strides = uint64_t(g.kb | g.kt | g.vb | g.vt | g.gb | g.gt);
    auto rows = [&](unsigned bytes) {
        bool ok = strides * uint64_t(es) % bytes == 0;
        for (const void *p : in) ok = ok && reinterpret_cast<uintptr_t>(p) % bytes == 0;
        return ok;
    };
    bool pairs = g.D % 2 == 0;
    for (const void *p : out) pairs = pairs && reinterpret_cast<uintptr_t>(p) % unsigned(2 * es) == 0;
    for (const void *p : f32) pairs = pairs && reinterpret_cast<uintptr_t>(p) % 8 == 0;
    if (pairs && g.D * es % 16 == 0 && rows(16)) return kCopy16;
    return es == 4 || (pairs && rows(4)) ? kCopy4 : kCopyAny;
}

// Blocks of a cluster.  Their exchange costs more the more they are, a lack of warps
// too: none where the lanes alone keep the SMs busy (`enough` of them), else as many as
// make up to `blocks`, as far as there are tiles.  2048 steps, us:
//   lanes                32    64    96   128   160   192   256
//   bf16 forward, 1    24.3  24.2  24.6  24.6  42.9  43.3  43.9
//                 4    13.4  17.5  21.6  26.5  36.7  41.5  47.3
//                 8    10.8  15.5  23.5  29.0  36.7  42.2  54.2
//                16    10.5  20.1  29.0  37.8  48.9  58.0  74.9
//       backward, 1    41.5  41.6  42.7  43.7  75.6  75.8  76.2
//                 4    16.8  25.7  40.6  51.2  63.9  75.1  88.4
//                 8    16.2  30.4  44.6  58.6  71.8  82.4   107
//   fp32 forward, 1    38.6  38.6  39.7  40.6  64.7  65.1  65.9
//                 4    16.0  23.1  38.8  47.8  60.3  69.6  83.5
//                 8    14.3  27.6  42.6  55.7  67.2  78.6   101
//       backward, 1    55.4  56.4  57.0  58.3  98.7  99.7   115
//                 4    21.0  43.9  65.1  86.1   107   128   167
//                 8    35.0  63.5  89.0   114   140   165   220
// The forward in bf16 has two bands, the others one, which misses the fastest form just
// past a lane an SM (160 lanes: 75.6 in place of 63.9 backward in bf16, 64.7 in place of 60.3
// forward in fp32), and backward in fp32 at about 32 lanes, where an SM holds one block of
// a cluster and 256 blocks take two turns (35.0 in place of 21.0).
int cluster_of(int64_t lanes, int64_t steps, int enough, int blocks) {
    int c = 1;
    if (lanes >= enough) return c;
    while (c < kMaxCluster && c * kTile < steps && 2 * c * lanes <= blocks) c *= 2;
    return c;
}
template <typename T>
int fwd_cluster(int64_t lanes, int64_t steps) {
    if (sizeof(T) == 4) return cluster_of(lanes, steps, 76, 256);
    return cluster_of(lanes, steps, lanes <= 152 ? 108 : 228, 640);  // (a lane on most SMs, or two)
}

// A kernel's form, without a cluster and with one: warps, steps of a tile, bytes of shared memory.
struct Form {
    int warps, tile;
    size_t smem;
};
template <typename T, bool CL>
Form fwd_form() {
    constexpr int W = kFwdWarps<T, CL>, tile = kFwdTile<T, CL>;
    return {W, tile, sizeof(Exchange<W, CL>) + 2 * 2 * tile * 64 * sizeof(T)};
}
template <typename T, bool CL>
Form bwd_form() {
    constexpr int W = kBwdWarps;
    return {W, kTile, sizeof(Exchange<W, CL>) + sizeof(float4) * 2 * W * 32 + 2 * 3 * kTile * 64 * sizeof(T)};
}

template <typename F, typename C>
cudaError_t run(F *plain, C *clustered, Args &g, int64_t lanes, int cluster, Form f, cudaStream_t s) {
    g.cluster = cluster, g.tiles = int((int64_t(g.T) + f.tile - 1) / f.tile);
    const void *fn = cluster > 1 ? reinterpret_cast<const void *>(clustered) : reinterpret_cast<const void *>(plain);
    const cudaError_t e = ensure_smem_attr(fn, int(f.smem));
    if (e != cudaSuccess) return e;
    if (cluster > 1) return launch_cluster(clustered, lanes * cluster, f.warps * 32, f.smem, cluster, s, g);
    plain<<<unsigned(lanes), f.warps * 32, f.smem, s>>>(g);
    return cudaGetLastError();
}

Args args_of(const mgs_gated_shape &sh) {
    Args g = {};
    g.D = sh.D, g.T = int(sh.T), g.strips = int((sh.D + 63) / 64);
    g.kb = sh.gate_stride[0], g.kt = sh.gate_stride[1], g.vb = sh.value_stride[0], g.vt = sh.value_stride[1];
    return g;
}
template <typename T, bool POS>
cudaError_t fwd_go(const mgs_gated_shape &sh, Args &g, cudaStream_t s) {
    const int64_t lanes = sh.B * g.strips;
    const int cluster = fwd_cluster<T>(lanes, sh.T);
    auto go = [&](auto how) {
        return run(gated_fwd_kernel<T, POS, how.value, false>, gated_fwd_kernel<T, POS, how.value, true>, g, lanes, cluster,
                   cluster > 1 ? fwd_form<T, true>() : fwd_form<T, false>(), s);
    };
    const Copy how = copy_of(g, sizeof(T));
    if (how == kCopy16) return go(std::integral_constant<Copy, kCopy16>());
    if constexpr (sizeof(T) == 2)
        if (how == kCopyAny) return go(std::integral_constant<Copy, kCopyAny>());
    return go(std::integral_constant<Copy, kCopy4>());
}
template <typename T, bool POS>
cudaError_t bwd_go(const mgs_gated_shape &sh, Args &g, cudaStream_t s) {
    const int64_t lanes = sh.B * g.strips;
    const int cluster = cluster_of(lanes, sh.T, 76, 256);
    auto go = [&](auto how) {
        return run(gated_bwd_kernel<T, POS, how.value, false>, gated_bwd_kernel<T, POS, how.value, true>, g, lanes, cluster,
                   cluster > 1 ? bwd_form<T, true>() : bwd_form<T, false>(), s);
    };
    const Copy how = copy_of(g, sizeof(T));
    if (how == kCopy16) return go(std::integral_constant<Copy, kCopy16>());
    if constexpr (sizeof(T) == 2)
        if (how == kCopyAny) return go(std::integral_constant<Copy, kCopyAny>());
    return go(std::integral_constant<Copy, kCopy4>());
}
template <typename T, bool POS>
cudaError_t step_go(const mgs_gated_shape &sh, Args &g, float *state, const int32_t *slots, int64_t nslots,
                    cudaStream_t s) {
    g.kt = g.vt = 0;
    g.out = state;
    // in pairs: neighbours in one load each (single elements for fp32 rows that start at 4 bytes alone)
    const Copy how = copy_of(g, sizeof(T));
    auto *fn = how == kCopy16 || (how == kCopy4 && sizeof(T) == 2) ? gated_step_kernel<T, POS, true>
                                                                   : gated_step_kernel<T, POS, false>;
    fn<<<unsigned((sh.B * g.strips + 3) / 4), 128, 0, s>>>((const T *)g.gate, (const T *)g.value, state, slots, nslots,
                                                          (T *)g.h, sh.B, sh.D, g.strips, g.kb, g.vb);
    return cudaGetLastError();
}

}  // namespace

#define MGS_BY_TYPE(go, ...)                                                                              \
    (sh.dtype == MGS_BF16 ? (sh.positive ? go<bf16, true>(__VA_ARGS__) : go<bf16, false>(__VA_ARGS__))    \
                          : (sh.positive ? go<float, true>(__VA_ARGS__) : go<float, false>(__VA_ARGS__)))

cudaError_t launch_gated_fwd(const mgs_gated_shape &sh, const void *gate, const void *value, const float *h0, void *h,
                             float *hT, float *carries, const DevCtl &ctl, cudaStream_t s) {
    Args g = args_of(sh);
    g.ctl = ctl;
    g.gate = gate, g.value = value, g.in = h0, g.h = h, g.out = hT, g.carries = carries;
    return MGS_BY_TYPE(fwd_go, sh, g, s);
}
cudaError_t launch_gated_bwd(const mgs_gated_shape &sh, const void *gate, const void *value, const float *carries,
                             const void *gh, const float *ghT, void *dgate, void *dvalue, float *dh0,
                             const DevCtl &ctl, cudaStream_t s) {
    Args g = args_of(sh);
    g.ctl = ctl;
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

cudaError_t launch_exchange_check(int late_block, int late_round, uint64_t late_ns, int32_t *rounds, int32_t *wrong,
                                  const DevCtl &ctl, cudaStream_t s) {
    return launch_cluster(exchange_check_kernel, kCheckBlocks, kCheckWarps * 32, 0, kCheckBlocks, s, late_block, late_round,
                          late_ns, rounds, wrong, ctl);
}

}  // namespace mgs
