// Embedding: out[n] = scale W[token_n], and the table's gradient
//   dW[v] = scale * (the sum of grad[n] over the n with token_n = v).
// A token outside 0..V-1 has a row of zeros and no gradient.  Bound by memory: the
// forward reads each row that is met and writes N; the backward reads N rows and
// writes V.
//
// The backward sorts the places n by their tokens, so that each row of dW is summed
// by one warp in the places' order and written once:
//   1. one cluster sorts (a stable radix sort of 8 bits a pass, counts exchanged
//      through distributed shared memory);
//   2. a block on each SM: some of its warps write rows of zeros (those whose tokens
//      the block has not found in the text), from the start; the others wait for the
//      order, then take a chunk of the sorted places and 1 KB of their rows at a time
//      and sum the runs of one token that begin in it, into the next chunk where they
//      go on there; of a run that is longer (a frequent word) each chunk's part goes
//      to the workspace.  Memory writes alone at 4.9 TB/s, with the sums' reads
//      beside them at more: the zeros are not written in a kernel of their own;
//   3. the long runs' parts are joined, a block a run.
// No atomics on the sums: the order is that of the tokens alone.  32768 tokens of a
// text, 50000 x 2048 in bf16: forward 26 us, backward 71 (sort 19 beside the zeros, joins
// 7; with the zeros in a kernel beside the sort alone 96).  Past that text the one cluster's
// sort and every block's reading of all tokens grow with the text: 131072 tokens of 2048 206
// us backward, 524288 734, of 256 columns 92 and 346; and one token more than 32768, past
// what the sort keeps in registers, 75 in place of 72 (of 256 columns 46 and 41).  A token
// that is all of a text is joined by one block for 128 columns: 524288 of 256 975 us.
#include "mgs_cluster.cuh"
#include "mgs_launch.h"
#include "mgs_lm.h"
#include "mgs_num.cuh"

namespace mgs {
namespace {

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kBins = 256;
constexpr int kWindow = 32768;   // rows of dW that a block marks at a time (bits in shared memory)
constexpr unsigned kNone = 0xffffffffu;
constexpr unsigned kCluster = 8, kKeep = 4;  // blocks that sort; a warp's batches that it keeps in registers

// The row pieces: 16 bytes (VEC), or single elements, a lane's 32 apart
template <typename T, bool VEC>
struct Piece {
    static constexpr int V = VEC ? kVec<T> : 1;
    float v[V];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = 0.f;
    }
};
template <typename T, bool VEC>
struct Raw;
template <typename T>
struct Raw<T, true> {
    uint4 u;
    __device__ __forceinline__ void load(const T *p) { u = __ldg(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void load_shared(const void *p) { u = *static_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(Piece<T, true> &f) const { unpack(u, f.v); }
};
template <typename T>
struct Raw<T, false> {
    T u;
    __device__ __forceinline__ void load(const T *p) { u = *p; }
    __device__ __forceinline__ void load_shared(const void *p) { u = *static_cast<const T *>(p); }
    __device__ __forceinline__ void get(Piece<T, false> &f) const { f.v[0] = to_f(u); }
};
template <typename T>
__device__ __forceinline__ void put(T *p, const Piece<T, true> &f) {
    __stcs(reinterpret_cast<uint4 *>(p), pack(f.v));
}
template <typename T>
__device__ __forceinline__ void put(T *p, const Piece<T, false> &f) { *p = from_f<T>(f.v[0]); }

// A warp takes up to U pieces a lane of a row: segment `seg` of `nseg`.
template <typename I, typename T, bool VEC, int U>
__global__ void __launch_bounds__(256)
    embed_fwd_kernel(const I *__restrict__ tokens, const T *__restrict__ w, float scale, T *__restrict__ out, int64_t N,
                     int64_t V, int64_t D, int nseg) {
    constexpr int P = Piece<T, VEC>::V;
    const int lane = threadIdx.x & 31;
    const int64_t items = N * nseg, step = int64_t(gridDim.x) * 8;
    for (int64_t i = int64_t(blockIdx.x) * 8 + threadIdx.x / 32; i < items; i += step) {
        const int64_t n = i / nseg, d0 = (i % nseg) * (32 * U * P) + lane * P, v = int64_t(tokens[n]);
        const bool live = v >= 0 && v < V;
        Raw<T, VEC> raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (live && d0 + u * 32 * P < D) raw[u].load(w + v * D + d0 + u * 32 * P);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (d0 + u * 32 * P >= D) break;
            Piece<T, VEC> f;
            if (live) raw[u].get(f);
            else f.zero();
#pragma unroll
            for (int j = 0; j < P; ++j) f.v[j] = live ? f.v[j] * scale : 0.f;
            put(out + n * D + d0 + u * 32 * P, f);
        }
    }
}

struct SortArgs {
    const void *tokens;
    unsigned *keys[2], *places[2];  // pass p writes [p & 1]
    int N, V, passes;
};

// One cluster sorts (token, place) by token, places in order; a token outside
// 0..V-1 counts as V.  A warp has consecutive places, a block consecutive warps.  A
// warp's batches of 32 are read once (KEEP: as many as stay in registers) or twice.
template <typename I, int KEEP>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(SortArgs a, unsigned cluster) {
    __shared__ unsigned at[kSortWarps][kBins];  // a warp's count of each digit, then its next place of it
    __shared__ unsigned quarter[4][kBins];      // a digit's count in eight of the warps
    __shared__ unsigned total[kBins], sums[8];
    griddep_launch();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31, digit_of = t & 255, eighth = (t >> 8) * 8;
    const unsigned rank = cluster_rank();
    // whole batches of 32 a warp
    const int64_t batches = (int64_t(a.N) + int64_t(cluster) * kSortThreads - 1) / (int64_t(cluster) * kSortThreads);
    const int64_t first = (int64_t(rank) * kSortWarps + warp) * batches * 32 + lane;
    for (int pass = 0; pass < a.passes; ++pass) {
        const unsigned *keys = a.keys[(pass & 1) ^ 1], *places = a.places[(pass & 1) ^ 1];
        auto key_of = [&](int64_t i) -> unsigned {
            if (pass > 0) return __ldcg(keys + i);  // (written by other blocks: past L1)
            const int64_t v = int64_t(__ldg(static_cast<const I *>(a.tokens) + i));
            return v >= 0 && v < a.V ? unsigned(v) : unsigned(a.V);
        };
        auto place_of = [&](int64_t i) { return pass > 0 ? __ldcg(places + i) : unsigned(i); };
        const int shift = 8 * pass;
        for (int i = t; i < kSortWarps * kBins; i += kSortThreads) (&at[0][0])[i] = 0;
        unsigned key[KEEP > 0 ? KEEP : 1], place[KEEP > 0 ? KEEP : 1];
        if constexpr (KEEP > 0) {
#pragma unroll
            for (int i = 0; i < KEEP; ++i)
                if (i < batches && first + i * 32 < a.N) key[i] = key_of(first + i * 32), place[i] = place_of(first + i * 32);
        }
        __syncthreads();
        if constexpr (KEEP > 0) {
#pragma unroll
            for (int i = 0; i < KEEP; ++i)
                if (i < batches && first + i * 32 < a.N) atomicAdd(&at[warp][(key[i] >> shift) & 255u], 1u);
        } else {
#pragma unroll 4
            for (int64_t i = 0; i < batches; ++i)
                if (first + i * 32 < a.N) atomicAdd(&at[warp][(key_of(first + i * 32) >> shift) & 255u], 1u);
        }
        __syncthreads();
        unsigned mine = 0;  // of this thread's digit, in its eight warps
#pragma unroll
        for (int w = 0; w < 8; ++w) mine += at[eighth + w][digit_of];
        quarter[eighth / 8][digit_of] = mine;
        __syncthreads();
        if (t < kBins) total[t] = quarter[0][t] + quarter[1][t] + quarter[2][t] + quarter[3][t];
        cluster_arrive();
        cluster_wait();
        unsigned before = 0;  // what comes before this thread's warps' places of its digit: smaller digits,
        {                     // the blocks and the warps in front
            unsigned all = 0;
#pragma unroll
            for (unsigned r = 0; r < kCluster; ++r) {
                const unsigned c = r < cluster ? ld_dsmem_u32(&total[digit_of], r) : 0u;
                before += r < rank ? c : 0u;
                all += c;
            }
            if (pass + 1 == a.passes) cluster_arrive();  // (no block leaves while its counts are read)
            unsigned s = all;
#pragma unroll
            for (int m = 1; m < 32; m *= 2) {
                const unsigned x = __shfl_up_sync(0xffffffffu, s, m);
                if (lane >= m) s += x;
            }
            if (t < kBins && lane == 31) sums[warp] = s;
            before += s - all;
        }
        __syncthreads();
        for (int w = 0; w < (warp & 7); ++w) before += sums[w];
        for (int q = 0; q < eighth / 8; ++q) before += quarter[q][digit_of];
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const unsigned c = at[eighth + w][digit_of];
            at[eighth + w][digit_of] = before;
            before += c;
        }
        __syncthreads();
        auto scatter = [&](int64_t i, unsigned k, auto value) {
            const bool live = first + i * 32 < a.N;
            const unsigned digit = (k >> shift) & 255u;
            const unsigned same = __match_any_sync(0xffffffffu, live ? digit : kBins);
            unsigned pos = 0;
            if (live) pos = at[warp][digit] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (live && lane == __ffs(same) - 1) at[warp][digit] += __popc(same);
            __syncwarp();
            if (live) a.keys[pass & 1][pos] = k, a.places[pass & 1][pos] = value();
        };
        if constexpr (KEEP > 0) {
#pragma unroll
            for (int i = 0; i < KEEP; ++i)
                if (i < batches) scatter(i, key[i], [&] { return place[i]; });
        } else {
            for (int64_t i = 0; i < batches; ++i) {
                const int64_t n = first + i * 32;
                scatter(i, n < a.N ? key_of(n) : 0u, [&] { return place_of(n); });
            }
        }
        if (pass + 1 < a.passes) cluster_arrive();  // what was scattered is read, and the counts are made anew, by the next pass
        cluster_wait();
    }
}

constexpr int kSumWarps = 24, kFillWarps = 8;  // of a block, and those that write zeros first
constexpr int kRows = 8;                             // a summing warp's rows on their way

struct SumArgs {
    const void *tokens;
    const unsigned *keys, *places;
    const void *grad;
    void *dw;
    float *part;
    int64_t gs, D, items;
    float scale;
    int N, V, chunk, nseg, window;  // window: rows of dW that a block marks and fills at a time
};

// Rows of zeros, by `warps` warps: of lo .. hi - 1 those whose bit is not set
template <typename T>
__device__ __forceinline__ void fill_rows(const SumArgs &a, int64_t lo, int64_t hi, const unsigned *bits, int warps) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t row_bytes = a.D * int64_t(sizeof(T));
    for (int64_t v = lo + warp; v < hi; v += warps) {
        if (bits[(v - lo) >> 5] >> ((v - lo) & 31) & 1u) continue;
        // whole pieces of 16 bytes, and what lies before and behind them in two's
        const uintptr_t p = reinterpret_cast<uintptr_t>(a.dw) + uintptr_t(v * row_bytes), q = p + row_bytes;
        const uintptr_t from = (p + 15) & ~uintptr_t(15), to = q & ~uintptr_t(15);
#pragma unroll 4
        for (uintptr_t e = from + lane * 16; e < to; e += 512)
            __stcs(reinterpret_cast<uint4 *>(e), make_uint4(0u, 0u, 0u, 0u));
        const uintptr_t head = p + 2 * lane, tail = (to > from ? to : from) + 2 * lane;
        if (head < from && head < q) *reinterpret_cast<uint16_t *>(head) = 0;
        if (tail < q) *reinterpret_cast<uint16_t *>(tail) = 0;
    }
}

// What a warp has to know of the sorted places for one chunk: the chunk's own and the
// next one's (a lane each), and where the runs at its ends come from and go to.
struct Places {
    unsigned key, place, key2, place2;
    unsigned before, last_first, last_before, after;
    __device__ __forceinline__ void load(const SumArgs &a, int64_t item) {
        const int64_t i0 = item / a.nseg * a.chunk;
        const int lane = threadIdx.x & 31;
        auto at = [&](const unsigned *p, int64_t i, unsigned none) { return i >= 0 && i < a.N ? __ldcg(p + i) : none; };  // (of the kernel before)
        const bool in = lane < a.chunk && item < a.items;
        key = in ? at(a.keys, i0 + lane, kNone) : kNone, place = in ? at(a.places, i0 + lane, 0u) : 0u;
        key2 = in ? at(a.keys, i0 + a.chunk + lane, kNone) : kNone, place2 = in ? at(a.places, i0 + a.chunk + lane, 0u) : 0u;
        before = at(a.keys, i0 - 1, kNone), last_first = at(a.keys, i0 - a.chunk, kNone);
        last_before = at(a.keys, i0 - a.chunk - 1, kNone), after = at(a.keys, i0 + 2 * a.chunk, kNone);
    }
};

// A chunk's runs.  A run that begins in a chunk and ends in it or in the next one is
// the former's; a longer one is summed in parts, one of each chunk that it touches.
template <typename T, bool VEC, int U>
__device__ __forceinline__ void sum_chunk(const SumArgs &a, int64_t item, const Places &p, unsigned char *ring) {
    constexpr int P = Piece<T, VEC>::V;
    const T *__restrict__ grad = static_cast<const T *>(a.grad);
    T *__restrict__ dw = static_cast<T *>(a.dw);
    const int chunk = a.chunk, lane = threadIdx.x & 31;
    const int64_t c = item / a.nseg, d0 = (item % a.nseg) * (32 * U * P) + lane * P;
    const int n = __popc(__ballot_sync(0xffffffffu, p.key < unsigned(a.V)));  // places with a row: first in the order
    if (n == 0) return;
    const unsigned head = __shfl_sync(0xffffffffu, p.key, 0), tail = __shfl_sync(0xffffffffu, p.key, n - 1);
    const unsigned follow = __shfl_sync(0xffffffffu, p.key2, 0);
    int i = 0;
    bool head_part = false;  // the first run is a part of one that began in an earlier chunk
    if (p.before == head) {
        const int lead = __popc(__ballot_sync(0xffffffffu, p.key == head));
        const bool from_last = p.last_first != head || p.last_before != head;
        if (from_last && !(lead == chunk && follow == head)) i = lead;  // the last chunk's warp has it
        else head_part = true;
    }
    const bool on = n == chunk && follow == tail;               // the last run goes on in the next chunk
    const bool through = head_part && head == tail;             // ... and began before this one
    const bool tail_part = on && p.after == tail && !through;   // ... and goes on past the next one
    // its places in the next chunk, where it ends there
    const int extra = on && p.after != tail && !through ? __popc(__ballot_sync(0xffffffffu, p.key2 == tail)) : 0;
    const int end = n + extra;
    // a bit for each of the chunk's places that ends a run, or its part
    const unsigned next = __shfl_down_sync(0xffffffffu, p.key, 1);
    const unsigned stops = __ballot_sync(0xffffffffu, lane < n && (lane == n - 1 ? extra == 0 : next != p.key));
    Piece<T, VEC> acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) acc[u].zero();
    auto row_of = [&](int at) {  // (every lane asks)
        const unsigned pa = __shfl_sync(0xffffffffu, p.place, at & 31), pb = __shfl_sync(0xffffffffu, p.place2, (at - n) & 31);
        return grad + int64_t(at < n ? pa : pb) * a.gs + d0;
    };
    auto use = [&](int at, const Raw<T, VEC> (&raw)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            Piece<T, VEC> f;
            raw[u].get(f);
#pragma unroll
            for (int e = 0; e < P; ++e) acc[u].v[e] += f.v[e];
        }
        if (at < n ? !(stops >> at & 1u) : at != end - 1) return;
        const unsigned k = __shfl_sync(0xffffffffu, p.key, min(at, n - 1));
        const bool to_head = head_part && k == head, to_tail = tail_part && k == tail;
        float *parts = a.part + (2 * c + (to_head ? 0 : 1)) * a.D;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t d = d0 + u * 32 * P;
            if (d < a.D) {
                if (to_head || to_tail) {
#pragma unroll
                    for (int e = 0; e < P; ++e) parts[d + e] = acc[u].v[e];
                } else {
#pragma unroll
                    for (int e = 0; e < P; ++e) acc[u].v[e] *= a.scale;
                    put(dw + int64_t(k) * a.D + d, acc[u]);
                }
            }
            acc[u].zero();
        }
    };
    if constexpr (VEC || sizeof(T) == 4) {
        // a ring of kRows rows in shared memory; a lane reads what it has copied itself
        constexpr int BYTES = VEC ? 16 : 4;
        auto slot = [&](int at, int u) { return ring + ((at & (kRows - 1)) * U + u) * (32 * BYTES) + lane * BYTES; };
        auto copy = [&](int at) {
            const T *row = row_of(at);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (at >= end || d0 + u * 32 * P >= a.D) continue;
                if constexpr (VEC)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(slot(at, u))), "l"(row + u * 32 * P) : "memory");
                else
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(slot(at, u))), "l"(row + u * 32 * P) : "memory");
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        for (int j = 0; j < kRows - 1; ++j) copy(i + j);
        for (int at = i; at < end; ++at) {
            copy(at + kRows - 1);
            asm volatile("cp.async.wait_group %0;" ::"n"(kRows - 1) : "memory");
            Raw<T, VEC> raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) raw[u].load_shared(slot(at, u));  // (past D: whatever lies there, and goes nowhere)
            use(at, raw);
        }
    } else {  // bf16 that starts anywhere: eight rows at a time
        constexpr int AHEAD = 8;
        for (; i < end; i += AHEAD) {
            Raw<T, VEC> raw[AHEAD][U];
#pragma unroll
            for (int j = 0; j < AHEAD; ++j) {
                const T *row = row_of(i + j);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (i + j < end && d0 + u * 32 * P < a.D) raw[j][u].load(row + u * 32 * P);
            }
#pragma unroll
            for (int j = 0; j < AHEAD; ++j)
                if (i + j < end) use(i + j, raw[j]);
        }
    }
}

template <typename I, typename T, bool VEC, int U>
__global__ void __launch_bounds__(kSumWarps * 32) embed_sum_kernel(const __grid_constant__ SumArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];  // the rows' bits, the rings
    unsigned *bits = reinterpret_cast<unsigned *>(smem);
    const I *tokens = static_cast<const I *>(a.tokens);
    const int warp = threadIdx.x >> 5;
    griddep_launch();
    const int64_t step = int64_t(gridDim.x) * a.window;
    for (int64_t lo = int64_t(blockIdx.x) * a.window; lo < a.V; lo += step) {
        const int64_t hi = min64(a.V, lo + a.window);
        for (int i = threadIdx.x; i < (a.window + 31) / 32; i += kSumWarps * 32) bits[i] = 0;
        __syncthreads();
#pragma unroll 8
        for (int n = threadIdx.x; n < a.N; n += kSumWarps * 32) {
            const int64_t v = int64_t(__ldg(tokens + n));
            if (v >= lo && v < hi) atomicOr(&bits[(v - lo) >> 5], 1u << ((v - lo) & 31));
        }
        __syncthreads();
        if (lo + step < a.V) {
            fill_rows<T>(a, lo, hi, bits, kSumWarps);
            __syncthreads();
        } else if (warp < kFillWarps) {  // the last rows: beside the sums
            fill_rows<T>(a, lo, hi, bits, kFillWarps);
        }
    }
    if (warp < kFillWarps) return;
    griddep_wait();
    constexpr int SUMS = kSumWarps - kFillWarps;
    unsigned char *ring = smem + kWindow / 8 + (warp - kFillWarps) * (kRows * 32 * U * Piece<T, VEC>::V * int(sizeof(T)));
    int64_t item = int64_t(blockIdx.x) * SUMS + warp - kFillWarps;
    const int64_t apart = int64_t(gridDim.x) * SUMS;
    Places now, next;
    for (now.load(a, item); item < a.items; item += apart, now = next) {
        next.load(a, item + apart);
        sum_chunk<T, VEC, U>(a, item, now, ring);
    }
}

// Runs in parts.  A block looks at 16 chunks (which begin such a run?) for 128 columns;
// its eight warps add up a run's parts, each every eighth one.
constexpr int kJoinChunks = 16, kJoinCols = 128;
template <typename T>
__global__ void __launch_bounds__(256, 8)
    embed_join_kernel(const unsigned *__restrict__ keys, const float *__restrict__ part, float scale,
                      T *__restrict__ dw, int N, int V, int64_t D, int chunk) {
    __shared__ float joined[8][kJoinCols];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int64_t d0 = int64_t(blockIdx.y) * kJoinCols, chunks = (int64_t(N) + chunk - 1) / chunk;
    griddep_wait();
    auto key_at = [&](int64_t i) { return i >= 0 && i < N ? keys[i] : kNone; };
    bool begins = false;  // (every warp looks at the same chunks)
    unsigned token = kNone;
    if (lane < kJoinChunks) {
        const int64_t i0 = (int64_t(blockIdx.x) * kJoinChunks + lane) * chunk;
        token = key_at(i0 + chunk - 1);
        const unsigned far = key_at(i0 + 2 * chunk), head = key_at(i0), last = key_at(i0 - 1);
        begins = token < unsigned(V) && far == token && (head != token || last != token);
    }
    for (unsigned left = __ballot_sync(0xffffffffu, begins); left; left &= left - 1) {
        const int which = __ffs(left) - 1;
        const unsigned v = __shfl_sync(0xffffffffu, token, which);
        const int64_t c = int64_t(blockIdx.x) * kJoinChunks + which;
        int len = 0;  // the chunks after c that begin with the token
        for (;;) {
            const int64_t next = c + 1 + len + lane;
            const int more = __popc(__ballot_sync(0xffffffffu, next < chunks && keys[next * chunk] == v));
            len += more;
            if (more < 32) break;
        }
        // part 0 is c's tail, parts 1.. the heads of the chunks behind it
        float s[4] = {};
#pragma unroll 2
        for (int m = warp; m <= len; m += 8) {
            const float *row = part + (2 * (c + m) + (m == 0)) * D + d0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (d0 + lane + 32 * j < D) s[j] += __ldcg(row + lane + 32 * j);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) joined[warp][lane + 32 * j] = s[j];
        __syncthreads();
        if (t < kJoinCols && d0 + t < D) {
            float sum = joined[0][t];
#pragma unroll
            for (int w = 1; w < 8; ++w) sum += joined[w][t];
            dw[int64_t(v) * D + d0 + t] = from_f<T>(scale * sum);
        }
        __syncthreads();
    }
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <typename I, typename T, bool VEC, int U>
cudaError_t fwd_at(const void *tokens, const void *w, float scale, void *out, int64_t N, int64_t V, int64_t D,
                   cudaStream_t s) {
    const int64_t nseg = (D + 32 * U * Piece<T, VEC>::V - 1) / (32 * U * Piece<T, VEC>::V);
    const int64_t grid = min64((N * nseg + 7) / 8, 152 * 64);
    embed_fwd_kernel<I, T, VEC, U><<<unsigned(grid), 256, 0, s>>>((const I *)tokens, (const T *)w, scale, (T *)out, N, V,
                                                                 D, int(nseg));
    return cudaGetLastError();
}
template <typename I, typename T>
cudaError_t fwd_go(const void *tokens, const void *w, float scale, void *out, int64_t N, int64_t V, int64_t D,
                   cudaStream_t s) {
    if (al16(w) && al16(out) && D % kVec<T> == 0) return fwd_at<I, T, true, 4>(tokens, w, scale, out, N, V, D, s);
    return fwd_at<I, T, false, 8>(tokens, w, scale, out, N, V, D, s);
}

// Places a chunk: 32, and fewer where that would leave the GPU without work (by 512 columns a segment, bf16's;
// the segments of fp32 and of rows that start anywhere are narrower, so that theirs are cut finer than they need)
int chunk_of(int64_t N, int64_t D) {
    int c = 32;
    while (c > 4 && (N / c) * ((D + 511) / 512) < 4096) c /= 2;
    return c;
}

struct Space {
    size_t keys, part, all;  // offsets in bytes: four arrays of N from 0, the parts
};
Space space_of(int64_t N, int64_t D) {
    const size_t array = (size_t(N) * 4 + 255) / 256 * 256;
    const int64_t chunks = (N + chunk_of(N, D) - 1) / chunk_of(N, D);
    return {array, 4 * array, 4 * array + size_t(chunks) * 2 * size_t(D) * 4};
}

template <typename I, typename T>
cudaError_t bwd_go(const void *tokens, const void *grad, int64_t gs, float scale, void *dw, int64_t N, int64_t V,
                   int64_t D, void *ws, cudaStream_t s) {
    const Space sp = space_of(N, D);
    char *base = static_cast<char *>(ws);
    auto array = [&](int i) { return reinterpret_cast<unsigned *>(base + i * sp.keys); };
    SortArgs a;
    a.tokens = tokens;
    a.keys[0] = array(0), a.keys[1] = array(1), a.places[0] = array(2), a.places[1] = array(3);
    a.N = int(N), a.V = int(V), a.passes = 1;
    while (V >> (8 * a.passes)) ++a.passes;  // V itself is a key
    const unsigned cluster = N <= 2048 ? 1 : kCluster;
    auto *sort = N <= int64_t(cluster) * kSortThreads * kKeep ? embed_sort_kernel<I, kKeep> : embed_sort_kernel<I, 0>;
    cudaError_t e = launch_cluster(sort, cluster, kSortThreads, 0, int(cluster), s, a, cluster);
    if (e != cudaSuccess) return e;
    const unsigned *keys = a.keys[(a.passes - 1) & 1], *places = a.places[(a.passes - 1) & 1];
    float *part = reinterpret_cast<float *>(base + sp.part);
    const int chunk = chunk_of(N, D);
    const int64_t chunks = (N + chunk - 1) / chunk;
    auto sum = [&](auto *fn, int width) {
        SumArgs b;
        b.tokens = tokens, b.keys = keys, b.places = places, b.grad = grad, b.dw = dw, b.part = part;
        b.gs = gs, b.D = D, b.scale = scale, b.N = int(N), b.V = int(V), b.chunk = chunk;
        b.nseg = int((D + width - 1) / width), b.items = chunks * b.nseg;
        const int64_t sums = (b.items + kSumWarps - kFillWarps - 1) / (kSumWarps - kFillWarps), rows = (V + 31) / 32;
        const int64_t blocks = min64(152, sums > rows ? sums : rows);
        b.window = int(min64(kWindow, (V + blocks - 1) / blocks));
        const size_t rings = kWindow / 8 + size_t(kSumWarps - kFillWarps) * kRows * (width * sizeof(T));
        const cudaError_t err = ensure_smem_attr(reinterpret_cast<const void *>(fn), int(rings));
        if (err != cudaSuccess) return err;
        return launch_next(fn, unsigned(blocks), kSumWarps * 32, rings, s, true, b);
    };
    const bool vec = al16(grad) && al16(dw) && D % kVec<T> == 0 && gs % kVec<T> == 0;
    e = vec ? sum(embed_sum_kernel<I, T, true, 2>, 64 * kVec<T>) : sum(embed_sum_kernel<I, T, false, 4>, 128);
    if (e != cudaSuccess) return e;
    if (chunks < 3) return cudaSuccess;  // no run is past a chunk and the next
    return launch_next(embed_join_kernel<T>,
                       dim3(unsigned((chunks + kJoinChunks - 1) / kJoinChunks), unsigned((D + kJoinCols - 1) / kJoinCols)),
                       256, 0, s, true, keys, (const float *)part, scale, (T *)dw, int(N), int(V), D, chunk);
}

}  // namespace

cudaError_t launch_embed_fwd(int itype, int dtype, const void *tokens, const void *w, float scale, void *out,
                             int64_t N, int64_t V, int64_t D, cudaStream_t s) {
    auto *go = itype == MGS_I64 ? (dtype == MGS_BF16 ? fwd_go<int64_t, bf16> : fwd_go<int64_t, float>)
                                : (dtype == MGS_BF16 ? fwd_go<int32_t, bf16> : fwd_go<int32_t, float>);
    return go(tokens, w, scale, out, N, V, D, s);
}

size_t embed_bwd_workspace_bytes(int64_t N, int64_t, int64_t D) { return space_of(N, D).all; }

cudaError_t launch_embed_bwd(int itype, int dtype, const void *tokens, const void *grad, int64_t gs, float scale,
                             void *dw, int64_t N, int64_t V, int64_t D, void *ws, cudaStream_t s) {
    auto *go = itype == MGS_I64 ? (dtype == MGS_BF16 ? bwd_go<int64_t, bf16> : bwd_go<int64_t, float>)
                                : (dtype == MGS_BF16 ? bwd_go<int32_t, bf16> : bwd_go<int32_t, float>);
    return go(tokens, grad, gs, scale, dw, N, V, D, ws, s);
}

}  // namespace mgs
