// Embedding: out[n] = scale W[token_n], and the table's gradient
//   dW[v] = scale * (the sum of grad[n] over the n with token_n = v).
// A token outside 0..V-1 has a row of zeros and no gradient.  Bound by memory: the
// forward reads each row that is met and writes N; the backward reads N rows and
// writes V.
//
// The backward sorts the places n by their tokens, so that each row of dW is summed
// by one warp in the places' order and written once:
//   1. one cluster sorts (a stable radix sort of 8 bits a pass, counts exchanged
//      through distributed shared memory), while the other blocks write the rows of
//      zeros, whose tokens they have not found in the text;
//   2. a warp takes a chunk of the sorted places and 1 KB of their rows: it
//      sums the runs of one token that begin in its chunk, into the next chunk
//      where they go on there; of a run that is longer (a frequent word) each
//      chunk's part goes to the workspace;
//   3. those parts are joined, a warp a run, or a block where there are many.
// No atomics on the sums: the order is that of the tokens alone.
#include "mgs_cluster.cuh"
#include "mgs_lm.h"
#include "mgs_num.cuh"

namespace mgs {
namespace {

constexpr int kSortThreads = 1024, kSortWarps = kSortThreads / 32, kBins = 256;
constexpr int kWindow = 32768;   // rows of dW that a block marks at a time (bits in shared memory)
constexpr unsigned kNone = 0xffffffffu;

__device__ __forceinline__ unsigned ld_dsmem_u32(const unsigned *p, unsigned rank) {
    unsigned v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(dsmem_addr(p, rank)) : "memory");
    return v;
}

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
    __device__ __forceinline__ void load_once(const T *p) { u = __ldcs(reinterpret_cast<const uint4 *>(p)); }
    __device__ __forceinline__ void get(Piece<T, true> &f) const { unpack(u, f.v); }
};
template <typename T>
struct Raw<T, false> {
    T u;
    __device__ __forceinline__ void load(const T *p) { u = *p; }
    __device__ __forceinline__ void load_once(const T *p) { u = *p; }
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
    int N, V, passes, window;       // window: rows of dW that a block fills at a time
    void *dw;
    int64_t row_bytes;
};

// Rows of zeros: of the rows that this block looks after, those whose tokens do not occur
template <typename I>
__device__ void fill_rows(const SortArgs &a, unsigned block, unsigned blocks, unsigned *bits) {
    const I *tokens = static_cast<const I *>(a.tokens);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int64_t lo = int64_t(block) * a.window; lo < a.V; lo += int64_t(blocks) * a.window) {
        const int64_t hi = min64(a.V, lo + a.window);
        for (int i = threadIdx.x; i < (a.window + 31) / 32; i += kSortThreads) bits[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int n = threadIdx.x; n < a.N; n += kSortThreads) {
            const int64_t v = int64_t(__ldg(tokens + n));
            if (v >= lo && v < hi) atomicOr(&bits[(v - lo) >> 5], 1u << ((v - lo) & 31));
        }
        __syncthreads();
        for (int64_t v = lo + warp; v < hi; v += kSortWarps) {
            if (bits[(v - lo) >> 5] >> ((v - lo) & 31) & 1u) continue;
            // whole pieces of 16 bytes, and what lies before and behind them in two's
            const uintptr_t p = reinterpret_cast<uintptr_t>(a.dw) + uintptr_t(v * a.row_bytes), q = p + a.row_bytes;
            const uintptr_t from = (p + 15) & ~uintptr_t(15), to = q & ~uintptr_t(15);
            for (uintptr_t e = from + lane * 16; e < to; e += 512)
                __stcs(reinterpret_cast<uint4 *>(e), make_uint4(0u, 0u, 0u, 0u));
            const uintptr_t head = p + 2 * lane, tail = (to > from ? to : from) + 2 * lane;
            if (head < from && head < q) *reinterpret_cast<uint16_t *>(head) = 0;
            if (tail < q) *reinterpret_cast<uint16_t *>(tail) = 0;
        }
        __syncthreads();
    }
}

// The first cluster sorts (token, place) by token, places in order; a token outside
// 0..V-1 counts as V.  A warp has consecutive places, a block consecutive warps.
template <typename I>
__global__ void __launch_bounds__(kSortThreads) embed_sort_kernel(SortArgs a, unsigned cluster) {
    __shared__ unsigned at[kSortWarps][kBins];  // a warp's count of each digit, then its next place of it
    __shared__ unsigned total[kBins], sums[8];
    griddep_launch();
    if (blockIdx.x >= cluster) {
        fill_rows<I>(a, blockIdx.x - cluster, gridDim.x - cluster, &at[0][0]);
        return;
    }
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const unsigned rank = cluster_rank();
    // whole batches of 32 a warp
    const int64_t batches = (int64_t(a.N) + int64_t(cluster) * kSortThreads - 1) / (int64_t(cluster) * kSortThreads);
    const int64_t first = (int64_t(rank) * kSortWarps + warp) * batches * 32;
    for (int pass = 0; pass < a.passes; ++pass) {
        const unsigned *keys = a.keys[(pass & 1) ^ 1], *places = a.places[(pass & 1) ^ 1];
        auto key_of = [&](int64_t i) -> unsigned {
            if (pass > 0) return __ldcg(keys + i);  // (written by other blocks: past L1)
            const int64_t v = int64_t(__ldg(static_cast<const I *>(a.tokens) + i));
            return v >= 0 && v < a.V ? unsigned(v) : unsigned(a.V);
        };
        const int shift = 8 * pass;
        for (int i = t; i < kSortWarps * kBins; i += kSortThreads) (&at[0][0])[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int64_t i = 0; i < batches; ++i) {
            const int64_t n = first + i * 32 + lane;
            if (n < a.N) atomicAdd(&at[warp][(key_of(n) >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (t < kBins) {  // from counts to the warps' places within the block's
            unsigned s = 0;
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
                const unsigned c = at[w][t];
                at[w][t] = s;
                s += c;
            }
            total[t] = s;
        }
        cluster_arrive();
        cluster_wait();
        unsigned before = 0, all = 0;
        if (t < kBins) {
            for (unsigned r = 0; r < cluster; ++r) {
                const unsigned c = ld_dsmem_u32(&total[t], r);
                before += r < rank ? c : 0u;
                all += c;
            }
            unsigned s = all;  // the sum of the digits up to this one
#pragma unroll
            for (int m = 1; m < 32; m *= 2) {
                const unsigned x = __shfl_up_sync(0xffffffffu, s, m);
                if (lane >= m) s += x;
            }
            if (lane == 31) sums[warp] = s;
            before += s - all;
        }
        __syncthreads();
        if (t < kBins) {
            for (int w = 0; w < warp; ++w) before += sums[w];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) at[w][t] += before;
        }
        __syncthreads();
        for (int64_t i = 0; i < batches; ++i) {
            const int64_t n = first + i * 32 + lane;
            const bool live = n < a.N;
            const unsigned key = live ? key_of(n) : 0u, digit = (key >> shift) & 255u;
            const unsigned same = __match_any_sync(0xffffffffu, live ? digit : kBins);
            unsigned pos = 0;
            if (live) pos = at[warp][digit] + __popc(same & ((1u << lane) - 1u));
            __syncwarp();
            if (live && lane == __ffs(same) - 1) at[warp][digit] += __popc(same);
            __syncwarp();
            if (live) {
                a.keys[pass & 1][pos] = key;
                a.places[pass & 1][pos] = pass > 0 ? __ldcg(places + n) : unsigned(n);
            }
        }
        cluster_arrive();  // what was scattered is read, and the counts are made anew, by the next pass
        cluster_wait();
    }
}

// A chunk's runs.  A run that begins in a chunk and ends in it or in the next one is
// the former's; a longer one is summed in parts, one of each chunk that it touches.
template <typename T, bool VEC, int U>
__global__ void __launch_bounds__(256)
    embed_sum_kernel(const unsigned *__restrict__ keys, const unsigned *__restrict__ places,
                     const T *__restrict__ grad, int64_t gs, float scale, T *__restrict__ dw, float *__restrict__ part,
                     int N, int V, int64_t D, int chunk, int nseg, int64_t items) {
    constexpr int P = Piece<T, VEC>::V;
    const int lane = threadIdx.x & 31;
    griddep_launch();
    griddep_wait();
    const int64_t item = int64_t(blockIdx.x) * 8 + threadIdx.x / 32;
    if (item >= items) return;
    const int64_t c = item / nseg, i0 = c * chunk, d0 = (item % nseg) * (32 * U * P) + lane * P;
    auto key_at = [&](int64_t i) { return i >= 0 && i < N ? keys[i] : kNone; };
    // this chunk's places and the next one's
    const bool mine = lane < chunk && i0 + lane < N, next_ok = lane < chunk && i0 + chunk + lane < N;
    unsigned key = mine ? keys[i0 + lane] : kNone, place = mine ? places[i0 + lane] : 0u;
    unsigned key2 = next_ok ? keys[i0 + chunk + lane] : kNone, place2 = next_ok ? places[i0 + chunk + lane] : 0u;
    const unsigned before = key_at(i0 - 1), last_first = key_at(i0 - chunk), last_before = key_at(i0 - chunk - 1),
                   after = key_at(i0 + 2 * chunk);
    const int n = __popc(__ballot_sync(0xffffffffu, key < unsigned(V)));  // places with a row: first in the order
    if (n == 0) return;
    const unsigned head = __shfl_sync(0xffffffffu, key, 0), tail = __shfl_sync(0xffffffffu, key, n - 1);
    const unsigned follow = __shfl_sync(0xffffffffu, key2, 0);
    int i = 0;
    bool head_part = false;  // the first run is a part of one that began in an earlier chunk
    if (before == head) {
        const int lead = __popc(__ballot_sync(0xffffffffu, key == head));
        const bool from_last = last_first != head || last_before != head;
        if (from_last && !(lead == chunk && follow == head)) i = lead;  // the last chunk's warp has it
        else head_part = true;
    }
    const bool on = n == chunk && follow == tail;               // the last run goes on in the next chunk
    const bool on_far = on && after == tail;                    // ... and past it
    const bool tail_part = on_far && !(head_part && head == tail);
    // (a run through the whole chunk that began earlier is head_part; it ends nowhere here)
    const int extra = on && !on_far && !(head_part && head == tail)
                          ? __popc(__ballot_sync(0xffffffffu, key2 == tail)) : 0;
    const int end = n + extra;
    Piece<T, VEC> acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) acc[u].zero();
    constexpr int AHEAD = 4;
    for (; i < end; i += AHEAD) {
        Raw<T, VEC> raw[AHEAD][U];
        unsigned k[AHEAD + 1];
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            const int at = i + j, l = at < n ? at : at - n;
            const unsigned ka = __shfl_sync(0xffffffffu, key, l & 31), kb = __shfl_sync(0xffffffffu, key2, l & 31);
            const unsigned pa = __shfl_sync(0xffffffffu, place, l & 31), pb = __shfl_sync(0xffffffffu, place2, l & 31);
            k[j] = at < n ? ka : at < end ? kb : kNone;
            if (at < end) {
                const T *row = grad + int64_t(at < n ? pa : pb) * gs + d0;
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (d0 + u * 32 * P < D) raw[j][u].load_once(row + u * 32 * P);
            }
        }
        {
            const int at = i + AHEAD, l = at < n ? at : at - n;
            const unsigned ka = __shfl_sync(0xffffffffu, key, l & 31), kb = __shfl_sync(0xffffffffu, key2, l & 31);
            k[AHEAD] = at < n ? ka : at < end ? kb : kNone;
        }
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) {
            if (i + j >= end) break;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                Piece<T, VEC> f;
                if (d0 + u * 32 * P < D) {
                    raw[j][u].get(f);
#pragma unroll
                    for (int e = 0; e < P; ++e) acc[u].v[e] += f.v[e];
                }
            }
            if (k[j + 1] == k[j]) continue;
            const bool to_head = head_part && k[j] == head, to_tail = tail_part && k[j] == tail;
            float *parts = part + (2 * c + (to_head ? 0 : 1)) * D;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t d = d0 + u * 32 * P;
                if (d < D) {
                    if (to_head || to_tail) {
#pragma unroll
                        for (int e = 0; e < P; ++e) parts[d + e] = acc[u].v[e];
                    } else {
#pragma unroll
                        for (int e = 0; e < P; ++e) acc[u].v[e] *= scale;
                        put(dw + int64_t(k[j]) * D + d, acc[u]);
                    }
                }
                acc[u].zero();
            }
        }
    }
}

// Runs in parts.  A block looks at 64 chunks (which begin such a run?) for 128
// columns; a warp joins a run of up to 32 chunks, the block's eight a longer one.
constexpr int kJoinChunks = 64, kJoinCols = 128;
template <typename T>
__global__ void __launch_bounds__(256)
    embed_join_kernel(const unsigned *__restrict__ keys, const float *__restrict__ part, float scale,
                      T *__restrict__ dw, int N, int V, int64_t D, int chunk) {
    __shared__ int found[kJoinChunks], lens[kJoinChunks];
    __shared__ int count;
    __shared__ float joined[8][kJoinCols];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    griddep_wait();
    if (t == 0) count = 0;
    __syncthreads();
    auto key_at = [&](int64_t i) { return i >= 0 && i < N ? keys[i] : kNone; };
    if (t < kJoinChunks) {
        const int64_t c = int64_t(blockIdx.x) * kJoinChunks + t, i0 = c * chunk;
        const unsigned tail = key_at(i0 + chunk - 1);
        const bool begins = tail < unsigned(V) && key_at(i0 + 2 * chunk) == tail &&
                            (key_at(i0) != tail || key_at(i0 - 1) != tail);
        if (begins) found[atomicAdd(&count, 1)] = t;  // (in any order: each is joined by itself)
    }
    __syncthreads();
    const int n = count;
    if (n == 0) return;
    const int64_t d0 = int64_t(blockIdx.y) * kJoinCols;
    const int64_t chunks = (int64_t(N) + chunk - 1) / chunk;
    auto add = [&](int64_t c, int from, int to, int step, float (&s)[4]) {
        // parts 1..: the heads of chunks c + 1 ..; part 0 is c's tail
#pragma unroll 4
        for (int m = from; m < to; m += step) {
            const float *row = part + (2 * (c + m) + (m == 0)) * D + d0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (d0 + lane + 32 * j < D) s[j] += __ldcg(row + lane + 32 * j);
        }
    };
    auto write = [&](unsigned v, const float (&s)[4]) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (d0 + lane + 32 * j < D) dw[int64_t(v) * D + d0 + lane + 32 * j] = from_f<T>(scale * s[j]);
    };
    for (int r = warp; r < n; r += 8) {
        const int64_t c = int64_t(blockIdx.x) * kJoinChunks + found[r];
        const unsigned v = keys[c * chunk + chunk - 1];
        // the chunks after c that begin with the token
        const unsigned on = __ballot_sync(0xffffffffu, c + 1 + lane < chunks && keys[(c + 1 + lane) * chunk] == v);
        const int len = __popc(on);
        if (lane == 0) lens[r] = len;
        if (len == 32) continue;
        float s[4] = {};
        add(c, 0, len + 1, 1, s);
        write(v, s);
    }
    __syncthreads();
    for (int r = 0; r < n; ++r) {
        if (lens[r] != 32) continue;
        const int64_t c = int64_t(blockIdx.x) * kJoinChunks + found[r];
        const unsigned v = keys[c * chunk + chunk - 1];
        int len = 0;
        for (;;) {
            const int more = __syncthreads_count(c + 1 + len + t < chunks && keys[(c + 1 + len + t) * chunk] == v);
            len += more;
            if (more < 256) break;
        }
        float s[4] = {};
        add(c, warp, len + 1, 8, s);
#pragma unroll
        for (int j = 0; j < 4; ++j) joined[warp][lane + 32 * j] = s[j];
        __syncthreads();
        if (warp == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                for (int w = 1; w < 8; ++w) s[j] += joined[w][lane + 32 * j];
            write(v, s);
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

// Places a chunk: 32, and fewer where that would leave the GPU without work
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
    a.tokens = tokens, a.dw = dw, a.row_bytes = D * int64_t(sizeof(T));
    a.keys[0] = array(0), a.keys[1] = array(1), a.places[0] = array(2), a.places[1] = array(3);
    a.N = int(N), a.V = int(V), a.passes = 1;
    while (V >> (8 * a.passes)) ++a.passes;  // V itself is a key
    const unsigned cluster = N <= 2048 ? 1 : 8;
    const int64_t fillers = min64(144 - cluster, (V + 31) / 32);
    const int64_t blocks = (cluster + fillers + cluster - 1) / cluster * cluster;
    a.window = int(min64(kWindow, (V + (blocks - cluster) - 1) / (blocks - cluster)));
    cudaError_t e = launch_cluster(embed_sort_kernel<I>, blocks, kSortThreads, 0, int(cluster), s, a, cluster);
    if (e != cudaSuccess) return e;
    const unsigned *keys = a.keys[(a.passes - 1) & 1], *places = a.places[(a.passes - 1) & 1];
    float *part = reinterpret_cast<float *>(base + sp.part);
    const int chunk = chunk_of(N, D);
    const int64_t chunks = (N + chunk - 1) / chunk;
    auto sum = [&](auto *fn, int width) {
        const int64_t nseg = (D + width - 1) / width, items = chunks * nseg;
        return launch_next(fn, unsigned((items + 7) / 8), 256, 0, s, true, keys, places, (const T *)grad, gs, scale,
                           (T *)dw, part, int(N), int(V), D, chunk, int(nseg), items);
    };
    const bool vec = al16(grad) && al16(dw) && D % kVec<T> == 0 && gs % kVec<T> == 0;
    e = vec ? sum(embed_sum_kernel<T, true, 2>, 64 * kVec<T>) : sum(embed_sum_kernel<T, false, 4>, 128);
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
