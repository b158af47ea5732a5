// Linear attention's walk (AttnWalk) for bf16 on the tensor cores, chunk by
// chunk.  Within a chunk of C = 128 steps with state S on entry and G_i the sum
// of g over the chunk's steps up to i (forward walk):
//   A   = Q K^T,   P_ij = A_ij e^{G_i - G_j} for j <= i, else 0
//   O   = diag(e^{G_i}) Q S + P V
//   S  <- e^{G_C} S + sum_j e^{G_C - G_j} k_j v_j^T
// and in reverse time (state S of the steps after the chunk)
//   P_ij = A_ij e^{G_j - G_i} for j >= i,   O = diag(e^{G_C - G_i}) Q S + P V
//   S  <- e^{G_C} S + sum_j e^{G_j} k_j v_j^T.
//
// The four products are 128 x 128 x 128 (tcgen05.mma, bf16, fp32 sums).  q, k
// and v are bf16 and enter exactly; what is computed enters as a sum of bf16
// terms: the weighted keys of the state always as three (24 bits: the state is
// fp32, and stays it), P and S as one where the output is rounded to bf16
// anyway, as three where <out, x> goes into the decay's gradient (TERMS).
//
// Heads of 64 go two to a block: panel p of a tile (64 columns) is head p; the
// state's product is formed for both at once and its two diagonal blocks used.
//
// Roles of the 18 warps (warp w reaches TMEM lanes 32 (w % 4) ..):
//   0..7   rows i of the chunk: P from A, the scaling of Q S, the output; warps
//          0..3 take columns 0..63, 4..7 columns 64..127
//   8..15  rows of the state (key index): the weighted keys, the state itself
//          in registers, the state as an operand; 8..11 and 12..15 share the
//          steps' groups and the state's columns
//   16     one thread issues the products
//   17     one thread loads tiles by TMA; the warp sums g
#include "mgs_launch.h"
#include "mgs_lm.h"
#include "mgs_num.cuh"
#include "mgs_tiles.cuh"
#include "mgs_umma.cuh"

#include <cudaTypedefs.h>

namespace mgs {
namespace {

constexpr int C = 128;
constexpr int kTile = 32768, kPanel = 16384;   // a tile: two panels of 128 rows x 64 bf16
constexpr int kThreads = 18 * 32;
constexpr int GT = 16;                         // steps of a group of weighted keys: one K = 16 product
constexpr int NG = C / GT;

// TMEM columns: A 0..127; P after it where it is one term, over it where it is three
constexpr uint32_t kA = 0, kO = 192, kKV = 320, kW = 448;
template <int TERMS>
constexpr uint32_t kP = TERMS == 1 ? 128 : 0;

template <int D, int TERMS>
struct Smem {
    static constexpr int NH = D == 64 ? 2 : 1;
    static constexpr int sterm = D == 64 ? kPanel : kTile;          // one term of the state operand
    static constexpr int NK = 2, NQ = TERMS == 1 ? 2 : 1, NV = TERMS == 1 || D == 64 ? 2 : 1;
    static constexpr int k = TERMS * sterm, q = k + NK * kTile, v = q + NQ * kTile, arr = v + NV * kTile;
    // per head: G (high and low parts), the column factors and the state weights of the 128 steps
    static constexpr int bars = arr + NH * 4 * C * 4;
    static constexpr size_t bytes = size_t(bars) + 256;
    static_assert(bytes <= 232448, "shared memory of an SM");
};

struct AttnMaps {
    CUtensorMap q[3], k[3], v[3];
};

__device__ __forceinline__ void mb_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int x, int y, int z, int w,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, "
        "%5}], [%6];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

// Waits for a phase; false once the wait gives up or another role has.
__device__ __noinline__ bool slow_wait(uint64_t *bar, uint32_t parity, volatile int *abort_word, DevCtl ctl) {
    const uint64_t t0 = global_ns();
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*abort_word != 0) return false;
        if (global_ns() - t0 > ctl.timeout_ns) {
            record_error(ctl, ERR_MBAR_TIMEOUT);
            *abort_word = 1;
            return false;
        }
    }
}

// x0, x1 as a sum of TERMS bf16 pairs (packed: x0 in the low half)
template <int TERMS>
__device__ __forceinline__ void split(float x0, float x1, uint32_t (&t)[TERMS]) {
    t[0] = pack_bf16(x0, x1);
#pragma unroll
    for (int i = 1; i < TERMS; ++i) {
        x0 -= bf_lo(t[i - 1]);
        x1 -= bf_hi(t[i - 1]);
        t[i] = pack_bf16(x0, x1);
    }
}

// (h, l) += (a, b), both sums of two fp32
__device__ __forceinline__ void add2(float &h, float &l, float a, float b) {
    const float s = h + a, t = s - h;
    const float e = (h - (s - t)) + (a - t);
    const float lo = l + b + e;
    h = s + lo;
    l = lo - (h - s);
}

template <int D, int TERMS>
__global__ void __launch_bounds__(kThreads, 1)
    attn_mma_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnSet set, int state_only) {
    using L = Smem<D, TERMS>;
    constexpr int NH = L::NH, SC = D == 64 ? 32 : 64;  // state columns of a thread
    extern __shared__ __align__(1024) unsigned char sm[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + L::bars);
    uint64_t *k_full = bars, *k_empty = bars + 2, *q_full = bars + 4, *q_empty = bars + 6, *v_full = bars + 8,
             *v_empty = bars + 10, *w_full = bars + 12, *w_empty = bars + 14;
    uint64_t *a_done = bars + 16, *p_ready = bars + 17, *qs_done = bars + 18, *o_done = bars + 19, *o_free = bars + 20,
             *s_ready = bars + 21, *kv_done = bars + 22, *kv_free = bars + 23, *g_full = bars + 24, *g_empty = bars + 25,
             *a_read = bars + 28, *drained = bars + 29;
    uint32_t *slot = reinterpret_cast<uint32_t *>(bars + 26);
    volatile int *abort_word = reinterpret_cast<volatile int *>(slot + 1);
    float *total = reinterpret_cast<float *>(slot + 2);  // [NH]: the chunk's decay

    const AttnWalk &w = set.w[blockIdx.y];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nseg = set.nseg, units = int((set.H + NH - 1) / NH);
    const int unit = int(blockIdx.x) / nseg, seg = int(blockIdx.x) - unit * nseg;
    const int b = unit / units, h0 = (unit - b * units) * NH;
    if (state_only && seg == (w.rev ? 0 : nseg - 1)) return;  // nothing starts from this segment's state
    const int H = int(set.H), T = int(set.T);
    const int c0 = int(seg * (set.seg_len / C)), c1 = min(c0 + int(set.seg_len / C), (T + C - 1) / C);
    const int n = c1 - c0;
    const bool rev = w.rev != 0;
    const DevCtl ctl = set.ctl;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 1), mbar_init(&q_full[i], 1), mbar_init(&v_full[i], 1);
            mbar_init(&k_empty[i], state_only ? 8 : 9);  // the readers of weighted keys, and Q K^T
            mbar_init(&q_empty[i], 1), mbar_init(&v_empty[i], 1);
            mbar_init(&w_full[i], 4), mbar_init(&w_empty[i], 1);
        }
        mbar_init(a_done, 1), mbar_init(p_ready, 8), mbar_init(qs_done, 1), mbar_init(o_done, 1), mbar_init(o_free, 8);
        mbar_init(s_ready, 8), mbar_init(kv_done, 1), mbar_init(kv_free, 8);
        mbar_init(g_full, 1), mbar_init(g_empty, state_only ? 8 : 16);
        mbar_init(a_read, 8), mbar_init(drained, 1);
        fence_barrier_init();
        *abort_word = (smem_addr(sm) & 1023u) != 0;  // the swizzled tiles need it (never seen otherwise)
    }
    if (warp == 16) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *slot;
    const uint32_t tq = tm + (uint32_t(32 * (warp & 3)) << 16);
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return mbar_try_wait(bar, parity & 1u) || slow_wait(bar, parity & 1u, abort_word, ctl);
    };
    // the same by a whole warp, whose lanes go on together
    auto wwait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    auto chunk_of = [&](int i) { return rev ? c1 - 1 - i : c0 + i; };
    const float *Gh = reinterpret_cast<const float *>(sm + L::arr);  // [NH][4][C]: G high, G low, column factor, weight
    const bool ok0 = *abort_word == 0;
    if (!ok0 && tid == 0) record_error(ctl, ERR_MBAR_TIMEOUT);

    if (!ok0) {
        // nothing was started
    } else if (warp < 8) {
        // ------------------------------------------------ rows of the chunk
        if (!state_only) {
            const int hh = warp >> 2, i = 32 * (warp & 3) + lane, wb = warp & 3;
            bool ok = true;
            for (int it = 0; it < n && ok; ++it) {
                const int c = chunk_of(it);
                const int64_t t = int64_t(c) * C + i;
                if (!(ok = wwait(g_full, it))) break;
                // weight of row i of Q S, for the head of this thread's output columns
                const float *Go = Gh + (NH == 2 ? hh * 4 * C : 0);
                const float ri = rev ? ex2_approx((Go[C - 1] - Go[i]) + (Go[2 * C - 1] - Go[C + i]))
                                     : ex2_approx(Go[i] + Go[C + i]);
                for (int hp = 0; hp < NH; ++hp) {
                    const float *G = Gh + hp * 4 * C;
                    const float gi = G[i], gl = G[C + i];
                    const int ev = it * NH + hp;
                    if (!(ok = wwait(a_done, ev))) break;
                    tc_fence_after();
                    // the product with the first head's P has read it
                    if (hp > 0 && !(ok = wwait(o_done, ev - 1))) break;
                    // two blocks of 32 columns j
                    float x[TERMS == 1 ? 1 : 2][32];
                    auto block_load = [&](int bl, float (&v)[32]) {
                        const int jb = 2 * hh + bl;
                        if (rev ? jb < wb : jb > wb) return;  // wholly masked
                        tmem_ld32(tq + kA + 32 * jb, v);
                        const float *cf = G + 2 * C + 32 * jb;
                        if (jb == wb) {
#pragma unroll
                            for (int u = 0; u < 32; u += 4) {
                                const float4 a = *reinterpret_cast<const float4 *>(G + 32 * jb + u);
                                const float4 l = *reinterpret_cast<const float4 *>(G + C + 32 * jb + u);
                                const float ah[4] = {a.x, a.y, a.z, a.w}, al[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                                for (int m = 0; m < 4; ++m) {
                                    const float e = (gi - ah[m]) + (gl - al[m]);
                                    const float f = ex2_approx(rev ? -e : e) * w.kv_scale;
                                    const bool in = rev ? u + m >= lane : u + m <= lane;
                                    v[u + m] = in ? v[u + m] * f : 0.f;
                                }
                            }
                        } else {
                            // off the diagonal the exponent splits at the block's edge between i
                            // and j, into a factor of the row and one of the column, neither above 1
                            const int ref = rev ? 32 * jb : 32 * jb + 31;
                            const float e = (gi - G[ref]) + (gl - G[C + ref]);
                            const float f = ex2_approx(rev ? -e : e) * w.kv_scale;
#pragma unroll
                            for (int u = 0; u < 32; u += 4) {
                                const float4 a = *reinterpret_cast<const float4 *>(cf + u);
                                v[u] *= f * a.x, v[u + 1] *= f * a.y, v[u + 2] *= f * a.z, v[u + 3] *= f * a.w;
                            }
                        }
                    };
                    if constexpr (TERMS == 1) {
#pragma unroll
                        for (int bl = 0; bl < 2; ++bl) {
                            uint32_t pk[16];
                            const int jb = 2 * hh + bl;
                            if (rev ? jb < wb : jb > wb) {
#pragma unroll
                                for (int u = 0; u < 16; ++u) pk[u] = 0u;
                            } else {
                                block_load(bl, x[0]);
#pragma unroll
                                for (int u = 0; u < 16; ++u) pk[u] = pack_bf16(x[0][2 * u], x[0][2 * u + 1]);
                            }
                            tmem_put16(tq + kP<TERMS> + 16 * jb, pk);
                        }
                    } else {
                        // P's terms take A's place: all of A is read before any is written
                        block_load(0, x[0]);
                        block_load(1, x[1]);
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mb_arrive(a_read);
                        if (!(ok = wwait(a_read, ev))) break;
                        tc_fence_after();
#pragma unroll
                        for (int bl = 0; bl < 2; ++bl) {
                            const int jb = 2 * hh + bl;
                            const bool none = rev ? jb < wb : jb > wb;
#pragma unroll
                            for (int half = 0; half < 2; ++half) {
                                uint32_t pk[TERMS][8];
#pragma unroll
                                for (int u = 0; u < 8; ++u) {
                                    uint32_t s[TERMS];
                                    split<TERMS>(x[bl][16 * half + 2 * u], x[bl][16 * half + 2 * u + 1], s);
#pragma unroll
                                    for (int m = 0; m < TERMS; ++m) pk[m][u] = none ? 0u : s[m];
                                }
#pragma unroll
                                for (int m = 0; m < TERMS; ++m)
                                    tmem_put8(tq + kP<TERMS> + 64 * m + 16 * jb + 8 * half, pk[m]);
                            }
                        }
                    }
                    tmem_wait_st();
                    if (hp == 0) {
                        // O = Q S scaled by rows, in place; P V is added to it
                        if (!(ok = wwait(qs_done, it))) break;
                        tc_fence_after();
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            float o[32];
                            tmem_ld32(tq + kO + 64 * hh + 32 * p, o);
#pragma unroll
                            for (int u = 0; u < 32; ++u) o[u] *= ri;
                            tmem_put32(tq + kO + 64 * hh + 32 * p, o);
                        }
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mb_arrive(p_ready);
                }
                if (!ok) break;
                if (lane == 0) mb_arrive(g_empty);
                // the output: row i, columns 64 hh ..
                const int h = NH == 2 ? h0 + hh : h0, col = NH == 2 ? 0 : 64 * hh;
                const bool live = t < T && h < H;
                uint4 xv[8];
                if (w.row_dot && live) {
                    const bf16 *px = static_cast<const bf16 *>(w.x) + b * w.xs[0] + t * w.xs[1] +
                                     (h / w.xdiv) * w.xs[2] + col;
#pragma unroll
                    for (int u = 0; u < 8; ++u) xv[u] = reinterpret_cast<const uint4 *>(px)[u];
                }
                if (!(ok = wwait(o_done, it * NH + NH - 1))) break;
                tc_fence_after();
                const int64_t at = b * w.os[0] + t * w.os[1] + h * w.os[2] + col;
                float dot = 0.f;
#pragma unroll
                for (int p = 0; p < 2; ++p) {
                    float o[32];
                    __syncwarp();
                    tmem_ld32(tq + kO + 64 * hh + 32 * p, o);
                    if (p == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mb_arrive(o_free);
                    }
#pragma unroll
                    for (int u = 0; u < 32; ++u) o[u] *= w.o_scale;
                    if (live && w.row_dot) {
#pragma unroll
                        for (int u = 0; u < 4; ++u) {
                            float xx[8];
                            unpack(xv[4 * p + u], xx);
#pragma unroll
                            for (int m = 0; m < 8; ++m) dot = fmaf(o[8 * u + m], xx[m], dot);
                        }
                    }
                    if (live && w.out_f32) {
                        float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(w.out) + at + 32 * p);
#pragma unroll
                        for (int u = 0; u < 8; ++u) to[u] = make_float4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
                    } else if (live) {
                        uint4 *to = reinterpret_cast<uint4 *>(static_cast<bf16 *>(w.out) + at + 32 * p);
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            to[u] = make_uint4(pack_bf16(o[8 * u], o[8 * u + 1]), pack_bf16(o[8 * u + 2], o[8 * u + 3]),
                                               pack_bf16(o[8 * u + 4], o[8 * u + 5]), pack_bf16(o[8 * u + 6], o[8 * u + 7]));
                    }
                }
                // heads of 128: each half of the columns leaves its own product
                if (w.row_dot && live)
                    w.row_dot[(NH == 2 ? 0 : hh * set.B * set.T * set.H) + (b * set.T + t) * set.H + h] = dot;
            }
        }
    } else if (warp < 16) {
        // ------------------------------------------------ rows of the state
        const int grp = (warp - 8) >> 2, dk = 32 * (warp & 3) + lane;
        const int hp = NH == 2 ? dk >> 6 : 0, h = h0 + hp;
        const int row = NH == 2 ? dk & 63 : dk, col = SC * grp;  // the head's state: row, first column
        const bool live = h < H;
        const int64_t ln = int64_t(b) * H + h;
        float s[SC];
        {
            const float *in = nullptr;
            bool tr = false;
            if (!state_only && live) {
                if (nseg > 1)
                    in = w.seg_in + (ln * nseg + seg) * D * D, tr = w.seg_t;
                else if (w.s_in)
                    in = w.s_in + ln * D * D, tr = w.s_in_t;
            }
#pragma unroll
            for (int u = 0; u < SC; ++u)
                s[u] = in == nullptr ? 0.f : tr ? in[(col + u) * D + row] : in[row * D + col + u];
        }
        auto put_state = [&](float *to, bool tr) {
            if (!live) return;
            if (tr) {
#pragma unroll
                for (int u = 0; u < SC; ++u) to[(col + u) * D + row] = s[u];
            } else {
#pragma unroll
                for (int u = 0; u < SC; u += 4)
                    *reinterpret_cast<float4 *>(to + row * D + col + u) = make_float4(s[u], s[u + 1], s[u + 2], s[u + 3]);
            }
        };
        auto checkpoint = [&](int c) {
            if (w.ckpt && ((c + 1) % (kAttnSpan / C) == 0 || (c + 1) * C >= T))
                put_state(w.ckpt + (ln * set.spans + c / (kAttnSpan / C)) * D * D, false);
        };
        // element (j, dk) of the keys' tile
        const uint32_t koff = uint32_t(dk >> 6) * kPanel + (dk & 7) * 2, kch = (dk & 63) >> 3;
        bool ok = true;
        for (int it = 0; it < n && ok; ++it) {
            const int c = chunk_of(it);
            if (rev) checkpoint(c);
            if (!state_only) {
                // the state as the operand of Q S (its reader of the chunk before is done)
                if (it > 0 && !(ok = wwait(qs_done, it - 1))) break;
                unsigned char *base = sm + (NH == 2 ? 0 : grp * kPanel) + dk * 128;
                const int ch0 = NH == 2 ? 4 * grp : 0;
#pragma unroll
                for (int u = 0; u < SC; u += 8) {
                    uint32_t t0[TERMS], t1[TERMS], t2[TERMS], t3[TERMS];
                    split<TERMS>(s[u], s[u + 1], t0);
                    split<TERMS>(s[u + 2], s[u + 3], t1);
                    split<TERMS>(s[u + 4], s[u + 5], t2);
                    split<TERMS>(s[u + 6], s[u + 7], t3);
#pragma unroll
                    for (int m = 0; m < TERMS; ++m)
                        *reinterpret_cast<uint4 *>(base + m * L::sterm + (((ch0 + u / 8) ^ (dk & 7)) << 4)) =
                            make_uint4(t0[m], t1[m], t2[m], t3[m]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mb_arrive(s_ready);
            }
            if (!(ok = wwait(&k_full[it % L::NK], it / L::NK) && wwait(g_full, it))) break;
            const unsigned char *kt = sm + L::k + (it % L::NK) * kTile + koff;
            const float *wt = Gh + hp * 4 * C + 3 * C;
            const float decay = total[hp];
            for (int i = 0; i < NG / 2 && ok; ++i) {
                const int gi = 2 * i + grp, use = it * (NG / 2) + i;
                uint32_t t[3][GT / 2];
#pragma unroll
                for (int u = 0; u < GT; u += 4) {
                    const float4 ww = *reinterpret_cast<const float4 *>(wt + gi * GT + u);
                    float x[4];
#pragma unroll
                    for (int m = 0; m < 4; ++m) {
                        const int j = gi * GT + u + m;
                        x[m] = __uint_as_float(
                            uint32_t(*reinterpret_cast<const uint16_t *>(kt + j * 128 + ((kch ^ (j & 7)) << 4))) << 16);
                    }
                    uint32_t a[3], d[3];
                    split<3>(x[0] * ww.x, x[1] * ww.y, a);
                    split<3>(x[2] * ww.z, x[3] * ww.w, d);
#pragma unroll
                    for (int m = 0; m < 3; ++m) t[m][u / 2] = a[m], t[m][u / 2 + 1] = d[m];
                }
                if (use > 0 && !(ok = wwait(&w_empty[grp], use - 1))) break;
                tc_fence_after();
#pragma unroll
                for (int m = 0; m < 3; ++m) tmem_put8(tq + kW + 24 * grp + 8 * m, t[m]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mb_arrive(&w_full[grp]);
            }
            if (!ok) break;
            if (lane == 0) mb_arrive(&k_empty[it % L::NK]), mb_arrive(g_empty);
            if (!(ok = wwait(kv_done, it))) break;
            tc_fence_after();
#pragma unroll
            for (int u = 0; u < SC; u += 32) {
                float x[32];
                tmem_ld32(tq + kKV + (NH == 2 ? 64 * hp : 0) + col + u, x);
#pragma unroll
                for (int m = 0; m < 32; ++m) s[u + m] = fmaf(decay, s[u + m], x[m]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mb_arrive(kv_free);
            if (!rev) checkpoint(c);
        }
        if (ok) {
            if (state_only)
                put_state(w.seg_out + (ln * nseg + seg) * D * D, w.seg_t);
            else if (w.s_out && seg == (rev ? 0 : nseg - 1))
                put_state(w.s_out + ln * D * D, false);
        }
    } else if (warp == 16) {
        // ------------------------------------------------ the products
        if (lane == 0) {
            constexpr uint32_t id_k = umma_idesc_bf16(128, 128, false), id_mn = umma_idesc_bf16(128, 128, true);
            constexpr uint32_t id_o = umma_idesc_bf16(128, D, true);
            const uint32_t sS = smem_addr(sm), sK = smem_addr(sm + L::k), sQ = smem_addr(sm + L::q),
                           sV = smem_addr(sm + L::v);
            auto qk = [&](int it, int hp) {
                const uint32_t q = sQ + (it % L::NQ) * kTile, k = sK + (it % L::NK) * kTile;
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                    const uint32_t off = uint32_t(NH == 2 ? hp : ks >> 2) * kPanel + uint32_t(ks & 3) * 32;
                    umma_bf16_ss(tm + kA, umma_desc_k(q + off), umma_desc_k(k + off), id_k, ks > 0);
                }
                umma_commit(a_done);
                if (hp == NH - 1) umma_commit(&k_empty[it % L::NK]);
            };
            auto qs = [&](int it) {
                const uint32_t q = sQ + (it % L::NQ) * kTile;
                for (int hp = 0; hp < NH; ++hp)
#pragma unroll
                    for (int m = 0; m < TERMS; ++m)
#pragma unroll
                        for (int ks = 0; ks < D / 16; ++ks) {
                            const uint32_t off = uint32_t(NH == 2 ? hp : ks >> 2) * kPanel + uint32_t(ks & 3) * 32;
                            umma_bf16_ss(tm + kO + 64 * hp, umma_desc_k(q + off),
                                         umma_desc_mn(sS + m * L::sterm + hp * 8192 + ks * 2048, kPanel), id_o,
                                         m + ks > 0);
                        }
                umma_commit(qs_done);
            };
            bool ok = true;
            for (int it = 0; it < n && ok; ++it) {
                if (!state_only) {
                    if (!(ok = wait(&k_full[it % L::NK], it / L::NK) && wait(&q_full[it % L::NQ], it / L::NQ))) break;
                    qk(it, 0);
                    if (!(ok = wait(s_ready, it) && (it == 0 || wait(o_free, it - 1)))) break;
                    tc_fence_after();
                    qs(it);
                    if (NH == 1) umma_commit(&q_empty[it % L::NQ]);
                }
                if (!(ok = wait(&v_full[it % L::NV], it / L::NV) && (it == 0 || wait(kv_free, it - 1)))) break;
                const uint32_t v = sV + (it % L::NV) * kTile;
                for (int gi = 0; gi < NG && ok; ++gi) {
                    const int buf = gi & 1;
                    if (!(ok = wait(&w_full[buf], it * (NG / 2) + (gi >> 1)))) break;
                    tc_fence_after();
#pragma unroll
                    for (int m = 0; m < 3; ++m)
                        umma_bf16_ts(tm + kKV, tm + kW + 24 * buf + 8 * m, umma_desc_mn(v + gi * 2048, kPanel), id_mn,
                                     gi + m > 0);
                    umma_commit(&w_empty[buf]);
                }
                if (!ok) break;
                umma_commit(kv_done);
                if (state_only) {
                    umma_commit(&v_empty[it % L::NV]);
                    continue;
                }
                for (int hp = 0; hp < NH && ok; ++hp) {
                    if (hp > 0) {
                        qk(it, hp);
                        umma_commit(&q_empty[it % L::NQ]);
                    }
                    if (!(ok = wait(p_ready, it * NH + hp))) break;
                    tc_fence_after();
#pragma unroll
                    for (int m = 0; m < TERMS; ++m)
#pragma unroll
                        for (int ks = 0; ks < C / 16; ++ks)
                            umma_bf16_ts(tm + kO + 64 * hp, tm + kP<TERMS> + 64 * m + 8 * ks,
                                         umma_desc_mn(v + hp * kPanel + ks * 2048, kPanel), id_o, true);
                    umma_commit(o_done);
                }
                if (ok) umma_commit(&v_empty[it % L::NV]);
            }
            // whatever was issued completes before TMEM and shared memory are released
            if (!ok) {
                umma_commit(drained);
                if (!mbar_wait_bounded(drained, 0, ctl.timeout_ns)) record_error(ctl, ERR_DRAIN_TIMEOUT);
            } else if (n > 0) {
                const bool done = mbar_wait_bounded(&v_empty[(n - 1) % L::NV], ((n - 1) / L::NV) & 1, ctl.timeout_ns);
                if (!done) record_error(ctl, ERR_DRAIN_TIMEOUT);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------ tiles and decays
        const float L2E = 1.4426950408889634f, L2E_LO = 1.9259629911266175e-8f;
        float *arr = reinterpret_cast<float *>(sm + L::arr);
        float gv[NH][4];
        auto fetch_g = [&](int c) {
#pragma unroll
            for (int hp = 0; hp < NH; ++hp)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int64_t t = int64_t(c) * C + 4 * lane + u;
                    gv[hp][u] = t < T && h0 + hp < H ? set.g[b * set.gs[0] + t * set.gs[1] + (h0 + hp) * set.gs[2]] : 0.f;
                }
        };
        if (n > 0) fetch_g(chunk_of(0));
        const CUtensorMap *mq = &maps.q[blockIdx.y], *mk = &maps.k[blockIdx.y], *mv = &maps.v[blockIdx.y];
        auto load = [&](unsigned char *dst, const CUtensorMap *m, int div, int c, uint64_t *full) {
            mbar_arrive_expect_tx(full, kTile);
#pragma unroll
            for (int p = 0; p < 2; ++p)
                tma_load_4d(dst + p * kPanel, m, NH == 2 ? 0 : 64 * p, c * C, (NH == 2 ? h0 + p : h0) / div, b, full);
        };
        // the next tile of a ring, once its slot is free
        auto fill = [&](int &l, int depth, uint64_t *full, uint64_t *empty, int off, const CUtensorMap *m, int div, int c) {
            const int sl = l % depth;
            if (l >= depth && !wait(&empty[sl], l / depth - 1)) return false;
            load(sm + off + sl * kTile, m, div, c, &full[sl]);
            ++l;
            return true;
        };
        bool ok = true;
        int lk = 0, lq = 0, lv = 0;  // tiles loaded
        for (int it = 0; it < n && ok; ++it) {
            const int c = chunk_of(it);
            // this warp runs about a chunk ahead: keys and queries, the sums of g once the
            // chunk before has used its own, then the values, whose tile is needed last
            if (lane == 0) {
                ok = fill(lk, L::NK, k_full, k_empty, L::k, mk, w.kdiv, c);
                if (!state_only) ok = ok && fill(lq, L::NQ, q_full, q_empty, L::q, mq, w.qdiv, c);
            }
            ok = __shfl_sync(0xffffffffu, int(ok), 0);
            if (!ok) break;
            // sums of g over the chunk, in units of log 2, as pairs of fp32
            float ph[NH][4], pl[NH][4];
#pragma unroll
            for (int hp = 0; hp < NH; ++hp) {
                float h = 0.f, l = 0.f;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float g = gv[hp][u];
                    float x = g * L2E;
                    float y = fmaf(g, L2E, -x) + g * L2E_LO;
                    if (x < -256.f) x = -256.f, y = 0.f;  // 2^-256 is 0 in fp32: so is any decay below
                    add2(h, l, x, y);
                    ph[hp][u] = h, pl[hp][u] = l;
                }
                float eh = h, el = l;  // inclusive sums over the lanes, then exclusive
#pragma unroll
                for (int m = 1; m < 32; m <<= 1) {
                    const float oh = __shfl_up_sync(0xffffffffu, eh, m), ol = __shfl_up_sync(0xffffffffu, el, m);
                    if (lane >= m) add2(eh, el, oh, ol);
                }
                eh = __shfl_up_sync(0xffffffffu, eh, 1), el = __shfl_up_sync(0xffffffffu, el, 1);
                if (lane == 0) eh = el = 0.f;
#pragma unroll
                for (int u = 0; u < 4; ++u) add2(ph[hp][u], pl[hp][u], eh, el);
            }
            if (it + 1 < n) fetch_g(chunk_of(it + 1));
            if (it > 0 && !(ok = wwait(g_empty, it - 1))) break;
#pragma unroll
            for (int hp = 0; hp < NH; ++hp) {
                float *G = arr + hp * 4 * C;
                const float lh = __shfl_sync(0xffffffffu, ph[hp][3], 31), ll = __shfl_sync(0xffffffffu, pl[hp][3], 31);
                // the edge of the 32-step block that column factors refer to
                const int src = (lane & 24) + (rev ? 0 : 7);
                const float rh = __shfl_sync(0xffffffffu, rev ? ph[hp][0] : ph[hp][3], src);
                const float rl = __shfl_sync(0xffffffffu, rev ? pl[hp][0] : pl[hp][3], src);
                float cf[4], wt[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float h = ph[hp][u], l = pl[hp][u];
                    cf[u] = exp2f(rev ? (h - rh) + (l - rl) : (rh - h) + (rl - l));
                    wt[u] = exp2f(rev ? h + l : (lh - h) + (ll - l)) * w.kv_scale;
                }
                store4(G + 4 * lane, ph[hp]);
                store4(G + C + 4 * lane, pl[hp]);
                store4(G + 2 * C + 4 * lane, cf);
                store4(G + 3 * C + 4 * lane, wt);
                if (lane == 31) total[hp] = exp2f(lh + ll);
                if (state_only && lane == 31 && h0 + hp < H) {
                    // the segment's sum of g beside its state, for the scan that joins the segments
                    float *sum = w.seg_out + set.B * set.H * nseg * D * D + (int64_t(b) * H + h0 + hp) * nseg + seg;
                    const float g = (lh + ll) * 0.6931471805599453f;
                    *sum = it == 0 ? g : *sum + g;
                }
            }
            __syncwarp();
            if (lane == 0) {
                mb_arrive(g_full);
                ok = fill(lv, L::NV, v_full, v_empty, L::v, mv, w.vdiv, c);
            }
            ok = __shfl_sync(0xffffffffu, int(ok), 0);
        }
        // every load in flight lands before the block's shared memory is released
        if (lane == 0) {
            bool done = true;
            for (int i = max(0, lk - L::NK); i < lk; ++i)
                done = mbar_wait_bounded(&k_full[i % L::NK], (i / L::NK) & 1, ctl.timeout_ns) && done;
            for (int i = max(0, lq - L::NQ); i < lq; ++i)
                done = mbar_wait_bounded(&q_full[i % L::NQ], (i / L::NQ) & 1, ctl.timeout_ns) && done;
            for (int i = max(0, lv - L::NV); i < lv; ++i)
                done = mbar_wait_bounded(&v_full[i % L::NV], (i / L::NV) & 1, ctl.timeout_ns) && done;
            if (!done) record_error(ctl, ERR_DRAIN_TIMEOUT);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// [B][T][heads][D] bf16 with any strides: boxes of 64 columns x 128 steps of one head
cudaError_t tile_map(CUtensorMap *m, const void *base, const int64_t (&st)[3], int64_t B, int64_t T, int64_t heads,
                     int D) {
    const uint64_t dims[4] = {uint64_t(D), uint64_t(T), uint64_t(heads), uint64_t(B)};
    // a dimension of one element is never stepped over: any legal stride does
    const uint64_t str[3] = {uint64_t(T > 1 ? st[1] : D) * 2, uint64_t(heads > 1 ? st[2] : D) * 2,
                             uint64_t(B > 1 ? st[0] : D) * 2};
    const uint32_t box[4] = {64, C, 1, 1};
    return make_tmap_bf16_4d(m, base, dims, str, box);
}

template <int D, int TERMS>
cudaError_t go(const AttnMaps &maps, const AttnSet &set, int nwalks, bool state_only, cudaStream_t s) {
    using L = Smem<D, TERMS>;
    const void *fn = (const void *)attn_mma_kernel<D, TERMS>;
    const cudaError_t e = ensure_smem_attr(fn, int(L::bytes));
    if (e != cudaSuccess) return e;
    const dim3 grid(unsigned(set.B * ((set.H + L::NH - 1) / L::NH) * set.nseg), unsigned(nwalks));
    attn_mma_kernel<D, TERMS><<<grid, kThreads, L::bytes, s>>>(maps, set, state_only);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_mma(const AttnSet &set, int nwalks, int D, int terms, bool state_only, cudaStream_t s) {
    AttnMaps maps;
    cudaError_t e;
    for (int i = 0; i < nwalks; ++i) {
        const AttnWalk &w = set.w[i];
        if ((e = tile_map(&maps.q[i], w.q, w.qs, set.B, set.T, set.H / w.qdiv, D)) != cudaSuccess) return e;
        if ((e = tile_map(&maps.k[i], w.k, w.ks, set.B, set.T, set.H / w.kdiv, D)) != cudaSuccess) return e;
        if ((e = tile_map(&maps.v[i], w.v, w.vs, set.B, set.T, set.H / w.vdiv, D)) != cudaSuccess) return e;
    }
    if (D == 64)
        return terms == 1 ? go<64, 1>(maps, set, nwalks, state_only, s) : go<64, 3>(maps, set, nwalks, state_only, s);
    return terms == 1 ? go<128, 1>(maps, set, nwalks, state_only, s) : go<128, 3>(maps, set, nwalks, state_only, s);
}

}  // namespace mgs
