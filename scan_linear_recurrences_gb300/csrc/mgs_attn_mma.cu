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
// fp32, and stays it); P and S as two (2^-17) where only the output's own rounding
// to bf16 follows, which is then the only one (with one term the output's error is
// 2.35e-3 instead of 1.66e-3 of it, for 128 us instead of 147 in the forward of 128
// lanes of 4096 steps), as three where <out, x> goes into the decay's gradient
// (TERMS).
//
// fp32 comes as three bf16 tensors whose sum it is, so that every operand has
// three terms and a product six pairs of them.  A block then has room for 64
// columns of a tile: a head of 128 is shared between two blocks, each with half
// of the state's columns (of the values and of the output), and a block takes
// q and k one half of their columns after the other, adding up A and Q S.
//
// Heads of 64 in bf16 go two to a block: panel p of a tile (64 columns) is head p; the
// state's product is formed for both at once and its two diagonal blocks used.
//
// Roles of the 20 warps (warp w reaches TMEM lanes 32 (w % 4) ..):
//   0..7   rows i of the chunk: P from A, the scaling of Q S, the output; warps
//          0..3 take columns 0..63, 4..7 columns 64..127
//   8..15  rows of the state (key index): the weighted keys, the state itself
//          in registers, the state as an operand; 8..11 and 12..15 share the
//          steps' groups and the state's columns
//   16     one thread issues the products
//   17     one thread loads tiles by TMA
//   18     sums of g
//   19     loads x; looks for infinities and NaN in v
//
// C = 128 is the products' M; shorter chunks would leave half of the tensor cores
// idle, longer ones need more TMEM than there is.  What bounds a block is the
// chain of a chunk: P from A (two thirds of the rows' time), the weighted keys'
// three terms (all of the state warps'), the products in their order between
// them.  A chunk takes 4.3 us of an SM (heads of 128 in bf16), 5.4 with three
// terms, 6.2 (two heads of 64), 6.2 and 9 (fp32, heads of 64 and 128); a block's
// start and end about 6 us.  152 lanes of 1024 steps, bf16, heads of 128: 45 us,
// 3.0 TB/s of HBM, tensor pipe 38 % (44 % with three terms; fp32 43 to 45 %; heads
// of 64 in bf16 25 %).
#include "mgs_launch.h"
#include "mgs_lm.h"
#include "mgs_num.cuh"
#include "mgs_tiles.cuh"
#include "mgs_umma.cuh"

#include <atomic>
#include <type_traits>

namespace mgs {
namespace {

constexpr int C = 128;
constexpr int kPanel = 16384;                  // a panel of a tile: 128 rows x 64 bf16
constexpr int kThreads = 20 * 32;              // five warpgroups
// Registers a thread: the kernel is launched with kRegs for each; the last
// warpgroup gives up what the others take more.  With heads of 128 and three
// terms the state's warps take some too (dq and dk of 128 lanes of 4096 steps 5
// us less); with two terms that costs the state-only walk more than it gives
// (1 x 16384 steps, 16 heads: 152 us against 124), with heads of 64 the last
// warpgroup's sums of g of two heads need the registers (717 us against 758).
constexpr int kRegs = 96, kRegsRows = 112;
template <int D, int TERMS, int IN>
struct Regs {
    static constexpr bool more = D == 128 && TERMS == 3 && IN == 1;
    static constexpr int state = more ? 104 : 96, last = more ? 48 : 64;
    static_assert(2 * kRegsRows + 2 * state + last <= 5 * kRegs, "within the registers of the launch");
};
constexpr int GT = 16;                         // steps of a group of weighted keys: one K = 16 product
constexpr int NG = C / GT;

// TMEM columns (all 512):
//   A 0..127, P over it (a third term behind it, to 191);
//   X 192..319: Q S, then (once the rows have it in registers) the state's product,
//   then (once that is in registers) P V;
//   the weighted keys of a chunk, three terms of 64 columns, 320..511.
struct Tmem {
    static constexpr uint32_t A = 0, P = 0, X = 192, O = 192, W = 320;
};

// mbarriers (of a ring: one a slot) and what goes with them
struct Bars {
    uint64_t k_full[2], k_empty[2], q_full[2], q_empty[2], v_full[2], v_empty[2];  // tiles
    uint64_t w_full[2], w_full2[2];                      // weighted keys, by halves of the chunk; of the second buffer
    uint64_t a_done, qs_done, o_done, kv_done, drained;  // products
    uint64_t p_ready, o_ready, o_free, s_ready, kv_free, st_sync;
    uint64_t g_full, g_empty, x_full, x_empty;
    uint64_t v_checked[4];
    int v_flag[4];                                       // the chunk's v has an infinity or NaN
    float total[2];                                      // the chunk's decay, of each head
    uint32_t slot;                                       // TMEM's address
};

template <int D, int TERMS, int IN>
struct Smem {
    static_assert(TERMS == 3 || (TERMS == 2 && IN == 1), "fp32: every operand in three terms");
    static constexpr int VD = IN == 3 ? 64 : D;                     // the state's columns in a block
    static constexpr int KH = IN == 3 ? D / 64 : 1;                 // passes over the columns of q and k
    static constexpr int NH = D == 64 && IN == 1 ? 2 : 1;           // heads of a block
    static constexpr int tile = IN == 1 ? 2 * kPanel : IN * kPanel;  // a tile: halves, heads or terms in its panels
    static constexpr int sterm = IN == 3 ? D * 128 : D == 64 ? kPanel : 2 * kPanel;  // a term of the state operand
    static constexpr int NK = TERMS == 2 ? 2 : 1, NQ = 1;  // (a second place for q gains nothing)
    static constexpr int NV = IN == 1 && (TERMS == 2 || D == 64) ? 2 : 1;
    static constexpr int k = TERMS * sterm, q = k + NK * tile, v = q + NQ * tile;
    // where rows are staged on their way out: with two terms the chunk's keys' place, else that of x
    static constexpr int x = v + NV * tile, arr = x + (TERMS == 2 ? 0 : 2 * kPanel);
    // per head: G (high and low parts), the column factors and the state weights of the 128 steps
    static constexpr int bars = arr + NH * 4 * C * 4;
    static constexpr int walk = bars + (sizeof(Bars) + 15) / 16 * 16;  // the block's AttnWalk
    static constexpr size_t bytes = size_t(walk) + sizeof(AttnWalk);
    static_assert(k % 1024 == 0, "swizzled tiles");
    static_assert(bytes <= 232448, "shared memory of an SM");
};

struct AttnMaps {
    CUtensorMap q[3], k[3], v[3], x[3], o[3];  // loads: 128 bytes x 128 steps; stores: x 32 steps
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

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// Tiled store shared -> global, a bulk group of the issuing thread; coordinates not negative
__device__ __forceinline__ void tma_store_4d(const CUtensorMap *map, int x, int y, int z, int w, const void *src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(src))
                 : "memory");
}
// 16 lanes x 8 columns: thread t holds, of lanes t / 4 and t / 4 + 8, column
// t % 4 in r[0], r[1] and column 4 + t % 4 in r[2], r[3]
__device__ __forceinline__ void tmem_put_16x8(uint32_t taddr, const uint32_t (&r)[4]) {
    asm volatile("tcgen05.st.sync.aligned.16x128b.x2.b32 [%0], {%1,%2,%3,%4};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3])
                 : "memory");
}

// One thread of a converged warp, of which the compiler knows that it is one.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}" : "=r"(p));
    return p != 0;
}

// Up to `tries` tries at a phase, in the fewest instructions: the waiting warps'
// tries take issue slots, and their code room in the instruction cache, from
// the working ones.  A try takes about 40 ns (84 cycles measured), so the limit
// counts tries instead of reading the clock.
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity, uint32_t tries) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, %3;\n\t"
        "AGAIN:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 q, n, 0;\n\t"
        "@q bra AGAIN;\n\t"
        "DONE:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(tries)
        : "memory");
    return ok != 0;
}

// x as a sum of TERMS bf16 pairs (packed: x.x in the low half)
template <int TERMS>
__device__ __forceinline__ void split(float2 x, uint32_t (&t)[TERMS]) {
    t[0] = pack_bf16(x.x, x.y);
#pragma unroll
    for (int i = 1; i < TERMS; ++i) {
        x = __ffma2_rn(make_float2(bf_lo(t[i - 1]), bf_hi(t[i - 1])), make_float2(-1.f, -1.f), x);
        t[i] = pack_bf16(x.x, x.y);
    }
}

// A row's part of P V alone: o += o_scale kv_scale sum_j e^(..) (q_t . k_j) v_j over
// the chunk's steps j on row t's side of the mask.  For chunks with an infinity
// or NaN among the v_j: the tensor cores multiply the masked entries too, and 0
// times it would reach the steps that v_j does not.
template <int D, int IN, int OC>
__device__ __forceinline__ void row_alone(const AttnWalk &w, const AttnSet &set, int b, int h, int t, int first, int end,
                                       int col, float *o) {
    const bf16 *q = static_cast<const bf16 *>(w.q) + b * w.qs[0] + t * w.qs[1] + (h / w.qdiv) * w.qs[2];
    const bf16 *k = static_cast<const bf16 *>(w.k) + b * w.ks[0] + (h / w.kdiv) * w.ks[2];
    const bf16 *v = static_cast<const bf16 *>(w.v) + b * w.vs[0] + (h / w.vdiv) * w.vs[2] + col;
    const float *g = set.g + b * set.gs[0] + h * set.gs[2];
    auto get = [](const bf16 *p, int64_t term, float (&x)[4]) {
        load4(p, x);
#pragma unroll
        for (int m = 1; m < IN; ++m) {
            float y[4];
            load4(p + m * term, y);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] += y[i];
        }
    };
    const int64_t qterm = set.B * w.qs[0], kterm = set.B * w.ks[0], vterm = set.B * w.vs[0];
    float sum = 0.f;  // of g between the row and step j
#pragma unroll 1
    for (int j = t; w.rev ? j < end : j >= first; j += w.rev ? 1 : -1) {
        if (w.rev && j > t) sum += g[j * set.gs[1]];
        float dot = 0.f, x[4], y[4];
#pragma unroll 1
        for (int c = 0; c < D; c += 4) {
            get(q + c, qterm, x), get(k + j * w.ks[1] + c, kterm, y);
#pragma unroll
            for (int i = 0; i < 4; ++i) dot = fmaf(x[i], y[i], dot);
        }
        const float p = dot * (w.o_scale * w.kv_scale * expf(sum));
        bool number = false;
#pragma unroll 1
        for (int c = 0; c < OC; c += 4) {
            get(v + j * w.vs[1] + c, vterm, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[c + i] = fmaf(p, x[i], o[c + i]);
                number = number || o[c + i] == o[c + i];
            }
        }
        if (!number) return;  // NaN throughout, and whatever comes leaves it so
        if (!w.rev) sum += g[j * set.gs[1]];
    }
}

// fp32: a product's second sum onto its first, 16 columns at a time
template <int N>
__device__ __forceinline__ void add_second(uint32_t taddr, float (&x)[N]) {
#pragma unroll
    for (int p = 0; p < N; p += 16) {
        float y[16];
        tmem_ld16(taddr + p, y);
#pragma unroll
        for (int u = 0; u < 16; u += 2) {
            const float2 z = __fadd2_rn(make_float2(x[p + u], x[p + u + 1]), make_float2(y[u], y[u + 1]));
            x[p + u] = z.x, x[p + u + 1] = z.y;
        }
    }
}

template <int D, int TERMS, int IN>
__global__ void __launch_bounds__(kThreads, 1)
    attn_mma_kernel(const __grid_constant__ AttnMaps maps, const __grid_constant__ AttnSet set, int state_only) {
    using L = Smem<D, TERMS, IN>;
    using M = Tmem;
    constexpr int NH = L::NH, KH = L::KH, VH = D / L::VD;
    constexpr int SC = L::VD / 2;               // state columns of a thread
    constexpr int OC = NH == 2 ? 64 : L::VD / 2;  // output columns of a thread
    extern __shared__ __align__(1024) unsigned char sm[];
    Bars &bars = *reinterpret_cast<Bars *>(sm + L::bars);
    uint64_t *k_full = bars.k_full, *k_empty = bars.k_empty, *q_full = bars.q_full, *q_empty = bars.q_empty,
             *v_full = bars.v_full, *v_empty = bars.v_empty, *w_full = bars.w_full, *w_full2 = bars.w_full2,
             *v_checked = bars.v_checked, *o_ready = &bars.o_ready, *st_sync = &bars.st_sync, *a_done = &bars.a_done,
             *p_ready = &bars.p_ready, *qs_done = &bars.qs_done, *o_done = &bars.o_done, *o_free = &bars.o_free,
             *s_ready = &bars.s_ready, *kv_done = &bars.kv_done, *kv_free = &bars.kv_free, *g_full = &bars.g_full,
             *g_empty = &bars.g_empty, *x_full = &bars.x_full, *x_empty = &bars.x_empty, *drained = &bars.drained;
    uint32_t *slot = &bars.slot;
    volatile int *v_flag = bars.v_flag;
    float *total = bars.total;

    // the walk's description from shared memory: parameters indexed by blockIdx
    // would be read through the global path
    const AttnWalk &w = *reinterpret_cast<const AttnWalk *>(sm + L::walk);
    const bool rev = set.w[set.first + blockIdx.y].rev != 0;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nseg = set.nseg, units = int((set.H + NH - 1) / NH) * VH;
    const int unit = int(blockIdx.x) / nseg, seg = int(blockIdx.x) - unit * nseg;
    const int b = unit / units, h0 = (unit - b * units) / VH * NH, v0 = (unit % VH) * L::VD;  // first head and column
    if (state_only && seg == (rev ? 0 : nseg - 1)) return;  // nothing starts from this segment's state
    const int H = int(set.H), T = int(set.T);
    const int c0 = int(seg * (set.seg_len / C)), c1 = min(c0 + int(set.seg_len / C), (T + C - 1) / C);
    const int n = c1 - c0;
    const DevCtl ctl = set.ctl;

    static_assert(sizeof(AttnWalk) % 4 == 0 && sizeof(AttnWalk) <= 4 * kThreads, "a word a thread");
    if (tid < int(sizeof(AttnWalk) / 4))
        reinterpret_cast<uint32_t *>(sm + L::walk)[tid] = reinterpret_cast<const uint32_t *>(&set.w[set.first + blockIdx.y])[tid];
    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&k_full[i], 1), mbar_init(&q_full[i], 1), mbar_init(&v_full[i], 1);
            // the rows' warps, who stage the output in it at the end, or its readers: the state's
            // warps and Q K^T
            mbar_init(&k_empty[i], TERMS == 2 || state_only ? 8 : 9);
            mbar_init(&q_empty[i], 1), mbar_init(&v_empty[i], state_only ? 1 : 2);
            mbar_init(&w_full[i], 8), mbar_init(&w_full2[i], 8);
        }
        mbar_init(a_done, 1), mbar_init(p_ready, 8), mbar_init(o_ready, 8), mbar_init(qs_done, 1), mbar_init(o_done, 1), mbar_init(o_free, 8);
        mbar_init(s_ready, 8), mbar_init(kv_done, 1), mbar_init(kv_free, 8);
        mbar_init(g_full, 1), mbar_init(g_empty, state_only ? 8 : 16);
        mbar_init(x_full, 1), mbar_init(x_empty, 8), mbar_init(drained, 1), mbar_init(st_sync, 8);
        for (int i = 0; i < 4; ++i) mbar_init(&v_checked[i], 1);
        fence_barrier_init();
    }
    if (warp == 16) {
        tmem_alloc(slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // What kernels of this call have written: fp32's terms are waited for here, bf16's states
    // below, where they are read (a kernel that runs beside this one may count on them too).
    if (IN == 3 || state_only) griddep_launch();
    if (IN == 3) griddep_wait();
    const uint32_t tm = *slot;
    const uint32_t tq = tm + (uint32_t(32 * (warp & 3)) << 16);
    // A role whose wait gives up says so and ends; the others' waits then give up too.
    const uint32_t tries = set.tries;
    auto wait = [&](uint64_t *bar, uint32_t parity) { return mbar_poll(smem_addr(bar), parity & 1u, tries); };
    // the same by a whole warp, whose lanes go on together
    auto wwait = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
    auto chunk_of = [&](int i) { return rev ? c1 - 1 - i : c0 + i; };
    const float *Gh = reinterpret_cast<const float *>(sm + L::arr);  // [NH][4][C]: G (-G in reverse) high and low, column factor, weight
    // the swizzled tiles need it (and have never been found elsewhere)
    const bool ok0 = (smem_addr(sm) & 1023u) == 0;
    if (!ok0 && tid == 0) record_error(ctl, ERR_MBAR_TIMEOUT);

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsRows));
        // ------------------------------------------------ rows of the chunk
        const int hh = warp >> 2, wb = warp & 3, i = 32 * wb + lane;
        const float kvs = w.kv_scale, os = w.o_scale;
        const int isgn = rev ? -1 : 1;
        const uint32_t in = rev ? ~0u << lane : ~0u >> (31 - lane);  // columns of the diagonal's block that count
        // the output's head, and the weights of its rows of Q S
        const int h = NH == 2 ? h0 + hh : h0, col = NH == 2 ? 0 : v0 + OC * hh;
        const float *Go = Gh + (NH == 2 ? hh * 4 * C : 0);
        bool ok = ok0;
#pragma unroll 1
        for (int it = 0; it < (state_only ? 0 : n) && ok; ++it) {
            const int c = chunk_of(it);
            if (!(ok = wwait(g_full, it))) break;
            float o1[OC];  // Q S, scaled by rows: the part of the output that comes from the state
            const float ri = os * ex2_approx(rev ? (Go[i] - Go[C - 1]) + (Go[C + i] - Go[2 * C - 1]) : Go[i] + Go[C + i]);
            auto from_state = [&]() {
                if (!wwait(qs_done, it)) return false;
                tc_fence_after();
#pragma unroll
                for (int p = 0; p < OC / 32; ++p) {
                    float x[32];
                    tmem_ld32(tq + M::X + OC * hh + 32 * p, x);
                    if (KH == 2) add_second(tq + M::X + 64 + OC * hh, x);
#pragma unroll
                    for (int u = 0; u < 32; u += 2) {
                        const float2 y = __fmul2_rn(make_float2(x[u], x[u + 1]), make_float2(ri, ri));
                        o1[32 * p + u] = y.x, o1[32 * p + u + 1] = y.y;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mb_arrive(o_ready);
                return true;
            };
            if (!(ok = from_state())) break;
            if (lane == 0 && it > 0) {  // the chunk before has been stored: its stage is free
                bulk_wait_read();
                mb_arrive(TERMS == 2 ? &k_empty[(it - 1) % L::NK] : x_empty);
            }
#pragma unroll 1
            for (int hp = 0; hp < NH; ++hp) {
                const float *G = Gh + hp * 4 * C;
                const float gi = G[i], gl = G[C + i];
                const int ev = it * NH + hp;
                if (!(ok = wwait(a_done, ev))) break;
                tc_fence_after();
                // the product with the first head's P has read it
                if (hp > 0 && !(ok = wwait(o_done, ev - 1))) break;
                // P from A, 16 columns j at a time.  Off the diagonal's block of 32 the
                // exponent splits at the block's edge between i and j, into a factor of the
                // row and one of the column, neither above 1; a block past it is zero.
                auto piece = [&](int j0, float (&v)[16]) {
                    const int jb = j0 >> 5;
                    if (isgn * (jb - wb) > 0) {
#pragma unroll
                        for (int u = 0; u < 16; ++u) v[u] = 0.f;
                        return;
                    }
                    tmem_ld16(tq + M::A + j0, v);
                    if (jb == wb) {
#pragma unroll
                        for (int u = 0; u < 16; u += 4) {
                            const float4 ah = *reinterpret_cast<const float4 *>(G + j0 + u);
                            const float4 al = *reinterpret_cast<const float4 *>(G + C + j0 + u);
                            const float e[4] = {(gi - ah.x) + (gl - al.x), (gi - ah.y) + (gl - al.y),
                                                (gi - ah.z) + (gl - al.z), (gi - ah.w) + (gl - al.w)};
#pragma unroll
                            for (int m = 0; m < 4; ++m) {
                                // computed whether or not it is masked: no branch for each element
                                const float y = v[u + m] * (ex2_approx(e[m]) * kvs);
                                v[u + m] = (in >> ((j0 & 31) + u + m)) & 1u ? y : 0.f;
                            }
                        }
                    } else {
                        const int ref = 32 * jb + (rev ? 0 : 31);
                        const float f = ex2_approx((gi - G[ref]) + (gl - G[C + ref])) * kvs;
#pragma unroll
                        for (int u = 0; u < 16; u += 4) {
                            const float4 a = *reinterpret_cast<const float4 *>(G + 2 * C + j0 + u);
                            const float2 ff = make_float2(f, f);
                            const float2 y = __fmul2_rn(make_float2(v[u], v[u + 1]), __fmul2_rn(ff, make_float2(a.x, a.y)));
                            const float2 z =
                                __fmul2_rn(make_float2(v[u + 2], v[u + 3]), __fmul2_rn(ff, make_float2(a.z, a.w)));
                            v[u] = y.x, v[u + 1] = y.y, v[u + 2] = z.x, v[u + 3] = z.y;
                        }
                    }
                };
                // The first two terms take the place of the 16 columns of A that this warp
                // has just read (nobody else touches them), a third has columns of its own.
#pragma unroll 1
                for (int j0 = 64 * hh; j0 < 64 * hh + 64; j0 += 16) {
                    float v[16];
                    piece(j0, v);
                    uint32_t pk[TERMS][8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        uint32_t t[TERMS];
                        split<TERMS>(make_float2(v[2 * u], v[2 * u + 1]), t);
#pragma unroll
                        for (int m = 0; m < TERMS; ++m) pk[m][u] = t[m];
                    }
                    tmem_put8(tq + M::P + j0, pk[0]);
                    tmem_put8(tq + M::P + j0 + 8, pk[1]);
                    if (TERMS == 3) tmem_put8(tq + M::P + 128 + j0 / 2, pk[TERMS - 1]);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mb_arrive(p_ready);
            }
            if (!ok) break;
            if (lane == 0) mb_arrive(g_empty);
            // The output: row i, this thread's columns.  The warp's 32 rows are staged (swizzled
            // rows of 128 bytes) where nobody else reads any more, two terms in the chunk's keys,
            // three in x's tile, and stored by TMA, which drops rows past the end.
            const int64_t tw = int64_t(c) * C + 32 * wb;  // the warp's first row
            unsigned char *stage = sm + (TERMS == 2 ? L::k + (it % L::NK) * L::tile : L::x) + hh * kPanel + 32 * wb * 128;
            unsigned char *mine = stage + lane * 128;
            const int live = h < H ? min(32, T - int(tw)) : 0;  // rows that exist (may be negative)
            auto own = [&](int u) { return reinterpret_cast<uint4 *>(mine + ((u ^ (lane & 7)) << 4)); };
            // (the answer for the fourth chunk from here waits for v's place, and that for the rows' P two
            // chunks on: it cannot overtake this wait)
            if (!(ok = wwait(&v_checked[it & 3], it >> 2) && wwait(o_done, it * NH + NH - 1))) break;
            if (__builtin_expect(v_flag[it & 3] != 0, 0)) {
                float o[OC];
#pragma unroll
                for (int u = 0; u < OC; ++u) o[u] = o1[u];
                if (lane < live) row_alone<D, IN, OC>(w, set, b, h, int(tw) + lane, c * C, min(c * C + C, T), col, o);
                __syncwarp();
#pragma unroll
                for (int u = 0; u < OC; ++u) o1[u] = o[u];
            } else {
                tc_fence_after();
#pragma unroll
                for (int p = 0; p < OC / 32; ++p) {
                    float o[32];
                    tmem_ld32(tq + M::O + OC * hh + 32 * p, o);
                    if (IN == 3) add_second(tq + M::O + 64 + OC * hh, o);
#pragma unroll
                    for (int u = 0; u < 32; u += 2) {
                        const float2 y = __ffma2_rn(make_float2(o[u], o[u + 1]), make_float2(os, os),
                                                    make_float2(o1[32 * p + u], o1[32 * p + u + 1]));
                        o1[32 * p + u] = y.x, o1[32 * p + u + 1] = y.y;
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mb_arrive(o_free);
            if (TERMS == 3 && w.row_dot) {
                constexpr int V = IN == 1 ? 8 : 4;
                if (!(ok = wwait(x_full, it))) break;
                float2 dot = make_float2(0.f, 0.f);
#pragma unroll
                for (int u = 0; u < 8; ++u) {  // a sum of short sums: half the rounding of one long one
                    float xx[V];
                    unpack(*own(u), xx);
                    float2 part = __fmul2_rn(make_float2(o1[V * u], o1[V * u + 1]), make_float2(xx[0], xx[1]));
#pragma unroll
                    for (int m = 2; m < V; m += 2)
                        part = __ffma2_rn(make_float2(o1[V * u + m], o1[V * u + m + 1]), make_float2(xx[m], xx[m + 1]), part);
                    dot = __fadd2_rn(dot, part);
                }
                __syncwarp();
                // a head in two warps, or in two of each of two blocks: each leaves its own product
                if (lane < live)
                    w.row_dot[(NH == 2 ? 0 : (v0 / OC + hh) * set.B * set.T * set.H) + (int64_t(b) * set.H + h) * set.T + tw + lane] =
                        dot.x + dot.y;
            }
            if (IN == 1 && w.out_f32) {
                // heads that share keys: each one's gradient in fp32, to be summed
                if (lane < live) {
                    float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(w.out) + b * w.os[0] +
                                                            (tw + lane) * w.os[1] + h * w.os[2] + col);
#pragma unroll
                    for (int u = 0; u < OC / 4; ++u)
                        to[u] = make_float4(o1[4 * u], o1[4 * u + 1], o1[4 * u + 2], o1[4 * u + 3]);
                }
            } else if constexpr (IN == 3) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    *reinterpret_cast<float4 *>(own(u)) =
                        make_float4(o1[4 * u], o1[4 * u + 1], o1[4 * u + 2], o1[4 * u + 3]);
            } else {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    *own(u) = make_uint4(pack_bf16(o1[8 * u], o1[8 * u + 1]), pack_bf16(o1[8 * u + 2], o1[8 * u + 3]),
                                         pack_bf16(o1[8 * u + 4], o1[8 * u + 5]), pack_bf16(o1[8 * u + 6], o1[8 * u + 7]));
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && (IN == 3 || !w.out_f32) && live > 0) tma_store_4d(&maps.o[blockIdx.y], col, int(tw), h, b, stage);
            if (lane == 0) bulk_commit();
        }
        if (!ok && lane == 0) record_error(ctl, ERR_MBAR_TIMEOUT);
        // the last chunks' tiles have been read before shared memory is released
        if (lane == 0) bulk_wait_read();
        __syncwarp();
    } else if (warp < 16) {
        if (Regs<D, TERMS, IN>::more)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<D, TERMS, IN>::state));
        // ------------------------------------------------ rows of the state
        const int grp = (warp - 8) >> 2, dk = 32 * (warp & 3) + lane;
        const int hp = NH == 2 ? dk >> 6 : 0, h = h0 + hp;
        const int row = NH == 2 ? dk & 63 : dk, col = SC * grp;  // the head's state: row, first column
        // heads of 64 in fp32: 64 key rows in 128 lanes, of which the upper half stands idle
        const bool mine = NH * D == 128 || dk < D, live = h < H && mine;
        const int64_t ln = int64_t(b) * H + h;
        float s[SC];
        // The state goes to and from memory 16 columns at a time through 2 KB of the warp's own
        // (the state operand's place, which is free whenever this is done): pieces of 64 bytes
        // of 8 rows instead of 16 bytes of 32.  Row r of the warp has its four 16-byte chunks
        // at c ^ (r / 2 % 4); thread t moves chunk t % 4 of rows t / 4, + 8, ..
        float4 *stage = reinterpret_cast<float4 *>(sm + (warp - 8) * 2048);
        auto at_row = [&](int c) { return stage + lane * 4 + (c ^ ((lane >> 1) & 3)); };
        auto at_line = [&](int j) { return stage + (8 * j + (lane >> 2)) * 4 + ((lane & 3) ^ ((lane >> 3) & 3)); };
        const int64_t moved = int64_t(row - lane + (lane >> 2)) * D + v0 + col + 4 * (lane & 3);
        {
            const float *in = nullptr;
            bool tr = false;
            if (IN == 1 && !set.beside) griddep_wait();
            if (IN == 1 && !state_only) griddep_launch();
            if (!state_only && live) {
                if (nseg > 1)
                    in = w.seg_in + (ln * nseg + seg) * D * D;
                else if (w.s_in)
                    in = w.s_in + ln * D * D, tr = w.s_in_t;
            }
            if (in == nullptr) {
#pragma unroll
                for (int u = 0; u < SC; ++u) s[u] = 0.f;
            } else if (tr) {
#pragma unroll
                for (int u = 0; u < SC; ++u) s[u] = in[(v0 + col + u) * D + row];
            } else {
#pragma unroll
                for (int u = 0; u < SC; u += 4) {  // piece u / 16, rows of j = u / 4 % 4
                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(in + moved + (u >> 4) * 16 + ((u >> 2) & 3) * 8 * D));
                    s[u] = x.x, s[u + 1] = x.y, s[u + 2] = x.z, s[u + 3] = x.w;
                }
#pragma unroll
                for (int u = 0; u < SC; u += 16) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        *at_line(j) = make_float4(s[u + 4 * j], s[u + 4 * j + 1], s[u + 4 * j + 2], s[u + 4 * j + 3]);
                    __syncwarp();
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 x = *at_row(j);
                        s[u + 4 * j] = x.x, s[u + 4 * j + 1] = x.y, s[u + 4 * j + 2] = x.z, s[u + 4 * j + 3] = x.w;
                    }
                    __syncwarp();
                }
            }
        }
        // no warp writes its rows of the operand into another's stage before that one is done
        uint32_t syncs = 0;
        auto staged = [&]() {
            __syncwarp();
            if (lane == 0) mb_arrive(st_sync);
            return wwait(st_sync, syncs++);
        };
        // The keys' tile is read transposed: ldmatrix gives thread t of a warp the
        // steps 2 (t % 4), + 1 of key row t / 4 (of 8 x 8 blocks), which is the
        // place of that pair in TMEM's 16-lane shape of 128 bits.  Address of this
        // thread's row of the four blocks (16 key rows x 16 steps):
        const int lr = ((lane >> 4) << 3) + (lane & 7);        // step within the group
        const int lc = ((32 * (warp & 3)) & 63) / 8 + ((lane >> 3) & 1);
        const uint32_t kbase = smem_addr(sm + L::k) + (IN == 1 ? (warp & 2) * (kPanel / 2) : 0) + lr * 128;
        const uint32_t kx0 = uint32_t((lc ^ (lr & 7)) << 4), kx1 = uint32_t(((lc + 2) ^ (lr & 7)) << 4);
        auto put_state = [&](float *to) {
#pragma unroll
            for (int u = 0; u < SC; u += 16) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *at_row(j) = make_float4(s[u + 4 * j], s[u + 4 * j + 1], s[u + 4 * j + 2], s[u + 4 * j + 3]);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) *reinterpret_cast<float4 *>(to + moved + u + j * 8 * D) = *at_line(j);
                __syncwarp();
            }
        };
        const bool marks = w.ckpt != nullptr;
        const int per_span = set.span / C;
        float decay = 0.f, next_decay = 0.f;  // of the chunk whose product is taken, and of the walked one
        bool ok = ok0 && staged();
#pragma unroll 1
        for (int it = 0; ok; ++it) {
            // States that are kept: at a span's end (in reverse that is the state before the
            // chunk is walked), and at the walk's end.
            if (!state_only) {
                const int ce = rev ? chunk_of(it) : chunk_of(it - 1);
                if (marks && (rev ? it < n : it > 0) && ((ce + 1) % per_span == 0 || (ce + 1) * C >= T) &&
                    ce / per_span < set.kept) {
                    if (live) put_state(w.ckpt + (ln * set.spans + ce / per_span) * D * D);
                    if (!(ok = staged())) break;
                }
                if (it == n) {
                    if (live && w.s_out && seg == (rev ? 0 : nseg - 1)) put_state(w.s_out + ln * D * D);
                    break;
                }
            }
            if (!state_only) {
                // the state as the operand of Q S (its reader of the chunk before is done)
                if (it > 0 && !(ok = wwait(qs_done, it - 1))) break;
                unsigned char *base = sm + (L::VD == 64 ? 0 : grp * kPanel) + dk * 128;
                const int ch0 = L::VD == 64 ? 4 * grp : 0;
                if (mine) {
#pragma unroll
                    for (int u = 0; u < SC; u += 8) {
                        uint32_t t0[TERMS], t1[TERMS], t2[TERMS], t3[TERMS];
                        split<TERMS>(make_float2(s[u], s[u + 1]), t0);
                        split<TERMS>(make_float2(s[u + 2], s[u + 3]), t1);
                        split<TERMS>(make_float2(s[u + 4], s[u + 5]), t2);
                        split<TERMS>(make_float2(s[u + 6], s[u + 7]), t3);
#pragma unroll
                        for (int m = 0; m < TERMS; ++m)
                            *reinterpret_cast<uint4 *>(base + m * L::sterm + (((ch0 + u / 8) ^ (dk & 7)) << 4)) =
                                make_uint4(t0[m], t1[m], t2[m], t3[m]);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mb_arrive(s_ready);
            }
            if (it < n) {
                if (!(ok = wwait(g_full, it))) break;
                const float *wt = Gh + hp * 4 * C + 3 * C + 2 * (lane & 3);
                next_decay = total[hp];
                if (!state_only) decay = next_decay;
                // the state-only walk has room for two chunks' keys, each with barriers of its own (it
                // makes the next chunk's before this one's have been asked for)
                const bool second = state_only && (it & 1);
                const uint32_t wcol = tq + (second ? M::A : M::W);
#pragma unroll 1
                for (int kh = 0; kh < KH; ++kh) {
                    const int kt_i = it * KH + kh;
                    if (!(ok = wwait(&k_full[kt_i % L::NK], kt_i / L::NK))) break;
                    const uint32_t kt = kbase + (kt_i % L::NK) * L::tile;
                    // the chunk's weighted keys, half of it at a time, the groups of 16 steps shared
                    // between the two warpgroups; a pass over half of the keys' columns is for the warps
                    // of those rows of the state
#pragma unroll 1
                    for (int i = KH == 1 || kh == ((warp & 3) >> 1) ? 0 : NG / 2; i < NG / 2; ++i) {
                        const int gi = (i >> 1) * (NG / 2) + grp * (NG / 4) + (i & 1);
                        const float2 w0 = *reinterpret_cast<const float2 *>(wt + gi * GT);
                        const float2 w1 = *reinterpret_cast<const float2 *>(wt + gi * GT + 8);
                        uint32_t r[2][4];  // key rows 0..15 and 16..31 of the warp
                        if (IN == 1) {
                            ldmatrix_x4_trans(kt + gi * (GT * 128) + kx0, r[0]);
                            ldmatrix_x4_trans(kt + gi * (GT * 128) + kx1, r[1]);
                        }
                        if (mine) {
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                uint32_t t[3][4], r1[4], r2[4];
                                if (IN == 3) {  // a key's three terms add up to it
                                    const uint32_t at = kt + gi * (GT * 128) + (x ? kx1 : kx0);
                                    ldmatrix_x4_trans(at, r[x]);
                                    ldmatrix_x4_trans(at + kPanel, r1);
                                    ldmatrix_x4_trans(at + 2 * kPanel, r2);
                                }
#pragma unroll
                                for (int m = 0; m < 4; ++m) {
                                    uint32_t a[3];
                                    float2 y = make_float2(bf_lo(r[x][m]), bf_hi(r[x][m]));
                                    if (IN == 3)
                                        y = __fadd2_rn(y, __fadd2_rn(make_float2(bf_lo(r1[m]), bf_hi(r1[m])),
                                                                     make_float2(bf_lo(r2[m]), bf_hi(r2[m]))));
                                    split<3>(__fmul2_rn(y, m < 2 ? w0 : w1), a);
                                    t[0][m] = a[0], t[1][m] = a[1], t[2][m] = a[2];
                                }
#pragma unroll
                                for (int m = 0; m < 3; ++m)
                                    tmem_put_16x8(wcol + (uint32_t(16 * x) << 16) + 64 * m + 8 * gi, t[m]);
                            }
                        }
                        if (i & 1) {
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mb_arrive(&(second ? w_full2 : w_full)[i >> 1]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0 && (state_only || TERMS == 3)) mb_arrive(&k_empty[kt_i % L::NK]);
                }
                if (!ok) break;
                if (lane == 0) mb_arrive(g_empty);
            }
            // the state-only walk makes the next chunk's keys before it takes this one's product
            const int j = state_only ? it - 1 : it;
            if (j >= 0) {
                if (!(ok = wwait(kv_done, j))) break;
                tc_fence_after();
#pragma unroll
                for (int u = 0; u < SC; u += 16) {
                    float x[16];
                    tmem_ld16(tq + M::X + (NH == 2 ? 64 * hp : 0) + col + u, x);
                    if (IN == 3) add_second(tq + M::X + 64 + col + u, x);
#pragma unroll
                    for (int m = 0; m < 16; m += 2) {
                        const float2 y = __ffma2_rn(make_float2(decay, decay), make_float2(s[u + m], s[u + m + 1]),
                                                    make_float2(x[m], x[m + 1]));
                        s[u + m] = y.x, s[u + m + 1] = y.y;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mb_arrive(kv_free);
            }
            decay = next_decay;
            if (state_only && it == n) {
                if (live) put_state(w.seg_out + (ln * nseg + seg) * D * D);
                break;
            }
        }
        if (!ok && lane == 0) record_error(ctl, ERR_MBAR_TIMEOUT);
    } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<D, TERMS, IN>::last));
    if (!ok0) {
        // nothing was started
    } else if (warp == 16) {
        // ------------------------------------------------ the products
        if (elect_one()) {
            // N: the steps; the state's columns (of both heads); a head's columns
            constexpr uint32_t id_k = umma_idesc_bf16(128, 128, false), id_mn = umma_idesc_bf16(128, NH * L::VD, true);
            constexpr uint32_t id_o = umma_idesc_bf16(128, L::VD, true);
            // Products of two sums of three terms: the pairs down to 2^-16 of the first,
            // (2,0) (1,1) (1,0) (0,2) (0,1) (0,0); a sum with an exact operand: its terms.  The
            // smallest first: the sums are cut off, not rounded, at each step, so that the fewest
            // steps should be made at full size.  For the same reason fp32's products over the 128
            // steps, and Q S with heads of 128, are two sums, added by who reads them.
            auto last = [](int m) { return IN == 1 ? 0 : 2 - m; };
            bool add = false;  // onto what is there
            // Descriptors hold addresses in units of 16 bytes: what is issued is one of these
            // plus a short sum, since longer ones between two products cost more time than a
            // product takes (64 cycles at N = 128).  Four steps' code in a row (fp32, B 16, T 1024: 90 us
            // against 100 in rolled loops); the loops around them are rolled, whose code stays at hand.
            const uint64_t dK = umma_desc_k(smem_addr(sm + L::k)), dQ = umma_desc_k(smem_addr(sm + L::q));
            const uint64_t dV = umma_desc_mn(smem_addr(sm + L::v), kPanel), dS = umma_desc_mn(smem_addr(sm), kPanel);
            constexpr int KS = D / 16 / KH;
            // K-major step ks of head hp: 32 bytes on in the rows, the next panel after four
            auto koff = [](int ks) { return uint64_t(((ks >> 2) * kPanel + (ks & 3) * 32) >> 4); };
            auto qk = [&](int it, int hp, int kh) {
                const int tile_i = it * KH + kh;
                const uint64_t q = dQ + uint64_t(((tile_i % L::NQ) * L::tile + hp * kPanel) >> 4);
                const uint64_t k = dK + uint64_t(((tile_i % L::NK) * L::tile + hp * kPanel) >> 4);
                add = kh > 0;
#pragma unroll 1
                for (int m = IN - 1; m >= 0; --m)
#pragma unroll 1
                    for (int o = last(m); o >= 0; --o)
#pragma unroll 4
                        for (int ks = 0; ks < KS; ++ks, add = true)
                            umma_bf16_ss(tm + M::A, q + koff(ks) + uint64_t(m * (kPanel >> 4)),
                                         k + koff(ks) + uint64_t(o * (kPanel >> 4)), id_k, add);
                if (kh == KH - 1) umma_commit(a_done);
                if (TERMS == 3 && hp == NH - 1) umma_commit(&k_empty[tile_i % L::NK]);
            };
            auto qs = [&](int it, int kh) {
                const int tile_i = it * KH + kh;
#pragma unroll 1
                for (int hp = 0; hp < NH; ++hp) {
                    const uint64_t q = dQ + uint64_t(((tile_i % L::NQ) * L::tile + hp * kPanel) >> 4);
                    add = false;
#pragma unroll 1
                    for (int m = TERMS - 1; m >= 0; --m) {
                        const uint64_t st = dS + uint64_t((m * L::sterm + (hp + kh) * 8192) >> 4);
#pragma unroll 1
                        for (int o = last(m); o >= 0; --o)
#pragma unroll 4
                            for (int ks = 0; ks < KS; ++ks, add = true)
                                umma_bf16_ss(tm + M::X + 64 * (hp + kh), q + koff(ks) + uint64_t(o * (kPanel >> 4)),
                                             st + uint64_t(ks * 128), id_o, add);
                    }
                }
                if (kh == KH - 1) umma_commit(qs_done);
            };
            // The state's product, half of the steps as soon as their keys are there; in one sum (IN = 1)
            // the largest terms come at the end, for both halves.
            auto kv = [&](int it, int half) {
                const uint64_t v = dV + uint64_t(((it % L::NV) * L::tile) >> 4);
                const uint32_t a = tm + (state_only && (it & 1) ? M::A : M::W);
                auto part = [&](int m, int o, int h) {
                    const uint32_t am = a + 64 * m + h * (NG / 2) * 8;
                    const uint64_t vo = v + uint64_t(h * (NG / 2) * 128 + o * (kPanel >> 4));
#pragma unroll 4
                    for (int i = 0; i < NG / 2; ++i, add = true)
                        umma_bf16_ts(tm + M::X + (IN == 3 ? 64 * h : 0), am + 8 * i, vo + uint64_t(i * 128), id_mn, add);
                };
                add = IN == 1 && half > 0;
#pragma unroll 1
                for (int m = 2; m >= (IN == 1 ? 1 : 0); --m)
#pragma unroll 1
                    for (int o = last(m); o >= 0; --o) part(m, o, half);
                if (IN == 1 && half == 1)
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) part(0, 0, h);
            };
            auto pv = [&](int it, int hp) {
                const uint64_t v = dV + uint64_t(((it % L::NV) * L::tile + hp * kPanel) >> 4);
                constexpr int KP = IN == 1 ? C / 16 : C / 32;  // steps of a sum
#pragma unroll 1
                for (int k0 = 0; k0 < C / 16; k0 += KP) {
                    add = false;
#pragma unroll 1
                    for (int m = TERMS - 1; m >= 0; --m) {
                        // 16 steps' first and second terms lie side by side, the third ones behind all
                        // of those
                        const uint32_t p = tm + M::P + (m == 2 ? 128 : 8 * m);
                        const uint32_t step = m == 2 ? 8 : 16;
#pragma unroll 1
                        for (int o = last(m); o >= 0; --o)
#pragma unroll 4
                            for (int ks = k0; ks < k0 + KP; ++ks, add = true)
                                umma_bf16_ts(tm + M::O + 64 * hp + (k0 > 0 ? 64 : 0), p + ks * step,
                                             v + uint64_t(ks * 128 + o * (kPanel >> 4)), id_o, add);
                    }
                }
                umma_commit(o_done);
            };
            bool ok = true;
#pragma unroll 1
            for (int it = 0; it < n && ok; ++it) {
                if (!state_only) {
                    // Q K^T at once: P has been made of the last one, and P's products are ahead of it in the
                    // queue
#pragma unroll 1
                    for (int kh = 0; kh < KH; ++kh) {
                        const int tile_i = it * KH + kh;
                        if (!(ok = wait(&q_full[tile_i % L::NQ], tile_i / L::NQ))) break;
                        if (!(ok = wait(&k_full[tile_i % L::NK], tile_i / L::NK))) break;
                        tc_fence_after();
                        qk(it, 0, kh);
                        if (kh == 0 && !(ok = wait(s_ready, it))) break;
                        if (kh == 0 && it > 0 && !(ok = wait(o_free, it - 1))) break;
                        tc_fence_after();
                        qs(it, kh);
                        if (NH == 1) umma_commit(&q_empty[tile_i % L::NQ]);
                    }
                    if (!ok || !(ok = wait(o_ready, it))) break;  // Q S is in the rows' registers
                } else if (it > 0 && !(ok = wait(kv_free, it - 1))) {
                    break;
                }
                uint64_t *keys = state_only && (it & 1) ? w_full2 : w_full;
                const uint32_t turn = state_only ? it >> 1 : it;
                if (!(ok = wait(&v_full[it % L::NV], it / L::NV) && wait(&keys[0], turn))) break;
                tc_fence_after();
                kv(it, 0);
                if (!(ok = wait(&keys[1], turn))) break;
                tc_fence_after();
                kv(it, 1);
                umma_commit(kv_done);
                if (!state_only) {
                    if (!(ok = wait(kv_free, it))) break;
                    if (!(ok = wait(p_ready, it * NH))) break;
                    tc_fence_after();
                    pv(it, 0);
                    if (NH == 2) {
                        qk(it, 1, 0);  // P stands over A: after the product with it
                        umma_commit(&q_empty[it % L::NQ]);
                        if (!(ok = wait(p_ready, it * NH + 1))) break;
                        tc_fence_after();
                        pv(it, 1);
                    }
                }
                umma_commit(&v_empty[it % L::NV]);
            }
            // whatever was issued completes before TMEM and shared memory are released
            if (!ok) {
                umma_commit(drained);
                record_error(ctl, wait(drained, 0) ? ERR_MBAR_TIMEOUT : ERR_MBAR_TIMEOUT | ERR_DRAIN_TIMEOUT);
            } else if (n > 0) {
                if (!wait(&v_empty[(n - 1) % L::NV], (n - 1) / L::NV)) record_error(ctl, ERR_DRAIN_TIMEOUT);
            }
        }
        __syncwarp();
    } else if (warp == 17) {
        // ------------------------------------------------ tiles
        if (lane == 0) {
            const CUtensorMap *mq = &maps.q[blockIdx.y], *mk = &maps.k[blockIdx.y], *mv = &maps.v[blockIdx.y];
            // the next tile of a ring, once its slot is free
            auto fill = [&](int i, int c, int depth, uint64_t *full, uint64_t *empty, int off, const CUtensorMap *m, int div,
                            int col) {
                const int sl = i % depth;
                if (i >= depth && !wait(&empty[sl], i / depth - 1)) return false;
                unsigned char *dst = sm + off + sl * L::tile;
                mbar_arrive_expect_tx(&full[sl], L::tile);
#pragma unroll 1
                for (int p = 0; p < L::tile / kPanel; ++p)  // halves of a head, heads, or terms (a batch apart)
                    tma_load_4d(dst + p * kPanel, m, NH * IN == 1 ? 64 * p : col, c * C, (NH == 2 ? h0 + p : h0) / div,
                                IN == 3 ? b + p * int(set.B) : b, &full[sl]);
                return true;
            };
            // a block starts with the state as an operand and Q, ends with V
            int lk = 0, lq = 0, lv = 0;  // tiles loaded
            bool ok = true;
#pragma unroll 1
            for (int it = 0; it < n && ok; ++it) {
                const int c = chunk_of(it);
#pragma unroll 1
                for (int kh = 0; kh < KH && ok; ++kh) {
                    if (!state_only) {
                        if (!(ok = fill(lq, c, L::NQ, q_full, q_empty, L::q, mq, w.qdiv, 64 * kh))) break;
                        ++lq;
                    }
                    if (!(ok = fill(lk, c, L::NK, k_full, k_empty, L::k, mk, w.kdiv, 64 * kh))) break;
                    ++lk;
                }
                if (!ok || !(ok = fill(lv, c, L::NV, v_full, v_empty, L::v, mv, w.vdiv, v0))) break;
                ++lv;
            }
            // every load in flight lands before the block's shared memory is released
            bool done = true;
            auto landed = [&](int l, int depth, uint64_t *full) {
#pragma unroll 1
                for (int i = max(0, l - depth); i < l; ++i) done = wait(&full[i % depth], i / depth) && done;
            };
            landed(lk, L::NK, k_full), landed(lq, L::NQ, q_full), landed(lv, L::NV, v_full);
            if (lv < n || !done) record_error(ctl, lv < n ? ERR_MBAR_TIMEOUT : ERR_DRAIN_TIMEOUT);
        }
        __syncwarp();
    } else if (warp == 18) {
        // ------------------------------------------------ decays
        const float L2E = 1.4426950408889634f, L2E_LO = 1.9259629911266175e-8f;  // log2(e) in two parts
        float *arr = reinterpret_cast<float *>(sm + L::arr);
        const float kvs = w.kv_scale;
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
        bool ok = true;
        if (n > 0) fetch_g(chunk_of(0));
#pragma unroll 1
        for (int it = 0; it < n && ok; ++it) {
            // sums of g over the chunk, in units of log 2, as pairs of fp32
            float ph[NH][4], pl[NH][4], cf[NH][4], wt[NH][4], last[NH];
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
#pragma unroll 1
                for (int m = 1; m < 32; m <<= 1) {
                    const float oh = __shfl_up_sync(0xffffffffu, eh, m), ol = __shfl_up_sync(0xffffffffu, el, m);
                    float th = eh, tl = el;
                    add2(th, tl, oh, ol);
                    eh = lane >= m ? th : eh, el = lane >= m ? tl : el;
                }
                eh = __shfl_up_sync(0xffffffffu, eh, 1), el = __shfl_up_sync(0xffffffffu, el, 1);
                if (lane == 0) eh = el = 0.f;
#pragma unroll
                for (int u = 0; u < 4; ++u) add2(ph[hp][u], pl[hp][u], eh, el);
                const float lh = __shfl_sync(0xffffffffu, ph[hp][3], 31), ll = __shfl_sync(0xffffffffu, pl[hp][3], 31);
                // the edge of the 32-step block that column factors refer to
                const int src = (lane & 24) + (rev ? 0 : 7);
                const float rh = __shfl_sync(0xffffffffu, rev ? ph[hp][0] : ph[hp][3], src);
                const float rl = __shfl_sync(0xffffffffu, rev ? pl[hp][0] : pl[hp][3], src);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const float h = ph[hp][u], l = pl[hp][u];
                    cf[hp][u] = ex2_approx(rev ? (h - rh) + (l - rl) : (rh - h) + (rl - l));
                    wt[hp][u] = ex2_approx(rev ? h + l : (lh - h) + (ll - l)) * kvs;
                    // the sign with which the rows' exponents come out as differences row - column
                    if (rev) ph[hp][u] = -h, pl[hp][u] = -l;
                }
                last[hp] = lh + ll;
            }
            if (it + 1 < n) fetch_g(chunk_of(it + 1));
            // the chunk before has used its own
            if (it > 0 && !(ok = wwait(g_empty, it - 1))) break;
#pragma unroll
            for (int hp = 0; hp < NH; ++hp) {
                float *G = arr + hp * 4 * C + 4 * lane;
                store4(G, ph[hp]);
                store4(G + C, pl[hp]);
                store4(G + 2 * C, cf[hp]);
                store4(G + 3 * C, wt[hp]);
                if (lane == 0) total[hp] = ex2_approx(last[hp]);
                if (state_only && lane == 0 && h0 + hp < H && v0 == 0) {
                    // the segment's sum of g beside its state, for the scan that joins the segments
                    float *sum = w.seg_out + set.B * set.H * nseg * D * D + (int64_t(b) * H + h0 + hp) * nseg + seg;
                    const float g = last[hp] * 0.6931471805599453f;
                    *sum = it == 0 ? g : *sum + g;
                }
            }
            __syncwarp();
            if (lane == 0) mb_arrive(g_full);
        }
        if (!ok && lane == 0) record_error(ctl, ERR_MBAR_TIMEOUT);
    } else if (!state_only) {
        // ------------------------------------------------ x, and whether all of v is finite
        constexpr int XN = IN == 1 ? 64 : 32;  // columns of a panel
        const bool has_x = TERMS == 3 && w.row_dot != nullptr;
        bool ok = true;
        int loads = 0;
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            // 0 times an infinity or NaN is NaN, and stays it in a sum (of three terms the first tells)
            if (!(ok = wwait(&v_full[it % L::NV], it / L::NV))) break;
            const uint4 *v = reinterpret_cast<const uint4 *>(sm + L::v + (it % L::NV) * L::tile) + lane;
            __nv_bfloat162 z[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) z[j] = __nv_bfloat162(bf16(0.f), bf16(0.f));
            const __nv_bfloat162 zero = z[0];
#pragma unroll 2
            for (int i = 0; i < (IN == 1 ? 2 : 1) * kPanel / 512; ++i) {
                const uint4 x = v[32 * i];
                z[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&x.x), zero, z[0]);
                z[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&x.y), zero, z[1]);
                z[2] = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&x.z), zero, z[2]);
                z[3] = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&x.w), zero, z[3]);
            }
            const __nv_bfloat162 sum = __hadd2(__hadd2(z[0], z[1]), __hadd2(z[2], z[3]));
            const bool bad = __any_sync(0xffffffffu, !(__low2float(sum) + __high2float(sum) == 0.f));
            if (lane == 0) {
                v_flag[it & 3] = bad;
                mb_arrive(&v_checked[it & 3]);
                mb_arrive(&v_empty[it % L::NV]);
            }
            if (has_x) {
                if (it > 0 && !(ok = wwait(x_empty, it - 1))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(x_full, 2 * kPanel);
#pragma unroll 1
                    for (int p = 0; p < 2; ++p)
                        tma_load_4d(sm + L::x + p * kPanel, &maps.x[blockIdx.y], NH == 2 ? 0 : v0 + XN * p,
                                    chunk_of(it) * C, (NH == 2 ? h0 + p : h0) / w.xdiv, b, x_full);
                }
                __syncwarp();
                ++loads;
            }
        }
        // the last load of x lands before the block's shared memory is released
        if (loads > 0) ok = wwait(x_full, loads - 1) && ok;
        if (!ok && lane == 0) record_error(ctl, ERR_MBAR_TIMEOUT);
    }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
    // what follows this kernel follows the one beside it too: one block's end is enough for that
    if (set.beside && blockIdx.x == gridDim.x - 1 && blockIdx.y == 0) griddep_wait();
}

// [B][T][heads][D] with any strides: boxes of 128 bytes x `steps` steps of one head
cudaError_t tile_map(CUtensorMap *m, const void *base, const int64_t (&st)[3], int64_t B, int64_t T, int64_t heads,
                     int D, int steps, bool f32) {
    const int es = f32 ? 4 : 2;
    const uint64_t dims[4] = {uint64_t(D), uint64_t(T), uint64_t(heads), uint64_t(B)};
    // a dimension of one element is never stepped over: any legal stride does
    const uint64_t str[3] = {uint64_t(T > 1 ? st[1] : D) * es, uint64_t(heads > 1 ? st[2] : D) * es,
                             uint64_t(B > 1 ? st[0] : D) * es};
    const uint32_t box[4] = {128u / es, uint32_t(steps), 1, 1};
    return make_tmap_4d(m, base, dims, str, box, f32);
}

template <int D, int TERMS, int IN>
cudaError_t go(const AttnMaps &maps, const AttnSet &set, int nwalks, bool state_only, bool early, cudaStream_t s) {
    using L = Smem<D, TERMS, IN>;
    const void *fn = (const void *)attn_mma_kernel<D, TERMS, IN>;
    cudaError_t e = ensure_smem_attr(fn, int(L::bytes));
    if (e != cudaSuccess) return e;
    // the split of the registers counts on this many at launch: with fewer the
    // warpgroups that ask for more would wait for good
    static std::atomic<int> regs{0};
    if (regs.load() == 0) {
        cudaFuncAttributes a;
        if ((e = cudaFuncGetAttributes(&a, fn)) != cudaSuccess) return e;
        regs.store(a.numRegs);
    }
    if (regs.load() != kRegs) return cudaErrorInvalidDeviceFunction;
    const dim3 grid(unsigned(set.B * ((set.H + L::NH - 1) / L::NH) * (D / L::VD) * set.nseg), unsigned(nwalks));
    return launch_next(attn_mma_kernel<D, TERMS, IN>, grid, kThreads, L::bytes, s, early, maps, set, int(state_only));
}

}  // namespace

cudaError_t launch_attn_mma(const AttnSet &all, int first, int nwalks, int D, int dtype, int terms, bool state_only,
                            bool early, bool beside, cudaStream_t s) {
    AttnMaps maps;
    AttnSet set = all;
    set.first = first, set.beside = beside;
    const bool f32 = dtype == MGS_F32;
    const int64_t B = set.B * (f32 ? 3 : 1);  // fp32 comes as three bf16 tensors behind one another
    cudaError_t e;
    for (int i = 0; i < nwalks; ++i) {
        const AttnWalk &w = set.w[first + i];
        if ((e = tile_map(&maps.q[i], w.q, w.qs, B, set.T, set.H / w.qdiv, D, C, false)) != cudaSuccess) return e;
        if ((e = tile_map(&maps.k[i], w.k, w.ks, B, set.T, set.H / w.kdiv, D, C, false)) != cudaSuccess) return e;
        if ((e = tile_map(&maps.v[i], w.v, w.vs, B, set.T, set.H / w.vdiv, D, C, false)) != cudaSuccess) return e;
        if (!state_only && w.row_dot &&
            (e = tile_map(&maps.x[i], w.x, w.xs, set.B, set.T, set.H / w.xdiv, D, C, f32)) != cudaSuccess)
            return e;
        if (!state_only && (f32 || !w.out_f32) &&
            (e = tile_map(&maps.o[i], w.out, w.os, set.B, set.T, set.H, D, 32, f32)) != cudaSuccess)
            return e;
    }
    auto *fn = f32 ? (D == 64 ? go<64, 3, 3> : go<128, 3, 3>)
               : D == 64 ? (terms == 2 ? go<64, 2, 1> : go<64, 3, 1>)
                         : (terms == 2 ? go<128, 2, 1> : go<128, 3, 1>);
    return fn(maps, set, nwalks, state_only, early || beside, s);
}

}  // namespace mgs
