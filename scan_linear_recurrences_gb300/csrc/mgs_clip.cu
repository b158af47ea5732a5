// The global norm of many tensors, and their scaling by it:
//   n = sqrt(sum over all elements of g^2),   out = g min(1, max_norm / (n + 1e-6)).
// Pass 1 leaves each block's sum of squares (fp32, of a fixed set of pieces in
// a fixed order); pass 2 adds those in every block, in the same order, and
// scales.  Bound by memory: every tensor is read twice and written once (2.2 GB
// of gradients: 317 us and 670 us, 7.0 and 6.6 TB/s, pass 2 from the end on, where
// the last of pass 1 is still in L2).  The
// tensors' addresses travel as kernel parameters, so the call copies nothing
// to the device and waits for nothing.
#include <cmath>

#include "mgs_lm.h"
#include "mgs_num.cuh"

namespace mgs {
namespace {

constexpr int kTensors = 512;      // tensors a launch (16 KB of the parameters)
constexpr int kPiece = 16384;      // elements of a piece
constexpr int kBlocks = 152 * 4;   // blocks of pass 1 a launch

struct ClipSet {
    const void *in[kTensors];
    void *out[kTensors];
    int64_t numel[kTensors];
    int first[kTensors + 1];       // index of a tensor's first piece; the last entry: all pieces
    uint8_t f32[kTensors];
    int count;
};
static_assert(sizeof(ClipSet) < 30000, "fits the kernel parameters");

// sum of squares, or the scaled copy, of elements [e0, e1) of a tensor
template <typename T, bool SCALE>
__device__ __forceinline__ float piece(const T *__restrict__ in, T *out, int64_t e0, int64_t e1, float c) {
    constexpr int V = kVec<T>;
    float sum = 0.f;
    const bool vec = ((reinterpret_cast<uintptr_t>(in) | (SCALE ? reinterpret_cast<uintptr_t>(out) : 0)) & 15u) == 0;
    int64_t e = e0;
    if (vec) {  // e0 is a multiple of kPiece
        const int64_t nv = (e1 - e0) / V;
        const uint4 *p = reinterpret_cast<const uint4 *>(in + e0);
        uint4 *o = reinterpret_cast<uint4 *>(out + e0);
        int64_t i = threadIdx.x;
        for (; i + 3 * blockDim.x < nv; i += 4 * blockDim.x) {
            uint4 u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) u[j] = p[i + j * blockDim.x];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v[V];
                unpack(u[j], v);
#pragma unroll
                for (int l = 0; l < V; ++l) {
                    if (SCALE)
                        v[l] *= c;
                    else
                        sum = fmaf(v[l], v[l], sum);
                }
                if (SCALE) o[i + j * blockDim.x] = pack(v);
            }
        }
        for (; i < nv; i += blockDim.x) {
            float v[V];
            unpack(p[i], v);
#pragma unroll
            for (int l = 0; l < V; ++l) {
                if (SCALE)
                    v[l] *= c;
                else
                    sum = fmaf(v[l], v[l], sum);
            }
            if (SCALE) o[i] = pack(v);
        }
        e = e0 + nv * V;
    }
    for (int64_t i = e + threadIdx.x; i < e1; i += blockDim.x) {
        const float x = to_f(in[i]);
        if (SCALE)
            out[i] = from_f<T>(x * c);
        else
            sum = fmaf(x, x, sum);
    }
    return sum;
}

template <bool SCALE>
__device__ __forceinline__ float pieces(const ClipSet &set, float c) {
    const int all = set.first[set.count];
    float sum = 0.f;
    for (int j = blockIdx.x; j < all; j += gridDim.x) {
        const int p = SCALE ? all - 1 - j : j;  // pass 2 backwards: what pass 1 read last is still in L2
        int lo = 0, hi = set.count;             // first[lo] <= p < first[hi]
        while (hi - lo > 1) {
            const int m = (lo + hi) / 2;
            if (set.first[m] <= p)
                lo = m;
            else
                hi = m;
        }
        const int64_t e0 = int64_t(p - set.first[lo]) * kPiece, e1 = min64(set.numel[lo], e0 + kPiece);
        if (set.f32[lo])
            sum += piece<float, SCALE>(static_cast<const float *>(set.in[lo]), static_cast<float *>(set.out[lo]), e0, e1, c);
        else
            sum += piece<bf16, SCALE>(static_cast<const bf16 *>(set.in[lo]), static_cast<bf16 *>(set.out[lo]), e0, e1, c);
    }
    return sum;
}

__device__ __forceinline__ float clip_block_sum(float x) {
    __shared__ float red[8];
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) x += __shfl_xor_sync(0xffffffffu, x, m);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[i];
    return t;
}

__global__ void __launch_bounds__(256) clip_sum_kernel(const __grid_constant__ ClipSet set, float *part) {
    const float s = clip_block_sum(pieces<false>(set, 0.f));
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__global__ void __launch_bounds__(256)
    clip_scale_kernel(const __grid_constant__ ClipSet set, const float *__restrict__ part, int nparts, float max_norm,
                      float *norm, bool write_norm) {
    float s = 0.f;
    for (int i = threadIdx.x; i < nparts; i += 256) s += part[i];
    s = sqrtf(clip_block_sum(s));
    if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = s;
    const float r = max_norm / (s + 1e-6f);
    // a NaN norm gives NaN (every element says so), as the formula does
    const float c = r >= 1.f ? 1.f : r;
    if (c == 1.f) {  // in place there is nothing to do; a copy is made of the tensors that have another target
        bool same = true;
        for (int i = 0; i < set.count; ++i) same = same && set.in[i] == set.out[i];
        if (same) return;
    }
    pieces<true>(set, c);
}

int64_t pieces_of(int64_t n) { return (n + kPiece - 1) / kPiece; }

}  // namespace

size_t clip_workspace_bytes(int64_t count) {
    const int64_t launches = count > 0 ? (count + kTensors - 1) / kTensors : 1;
    return size_t(launches) * kBlocks * sizeof(float);
}

cudaError_t launch_clip(const void *const *in, void *const *out, const int64_t *numel, const int32_t *dtypes,
                        int64_t count, float max_norm, float *norm, void *ws, cudaStream_t s) {
    float *part = static_cast<float *>(ws);
    const int64_t launches = count > 0 ? (count + kTensors - 1) / kTensors : 1;
    int nparts = 0;
    for (int pass = 0; pass < 2; ++pass) {
        for (int64_t l = 0; l < launches; ++l) {
            ClipSet set;
            const int64_t i0 = l * kTensors;
            set.count = int(min64(kTensors, count - i0));
            int64_t p = 0;
            for (int i = 0; i < set.count; ++i) {
                set.in[i] = in[i0 + i], set.out[i] = out[i0 + i], set.numel[i] = numel[i0 + i];
                set.f32[i] = dtypes[i0 + i] == MGS_F32;
                set.first[i] = int(p);
                p += pieces_of(numel[i0 + i]);
                if (p > 0x7fffffff - kBlocks) return cudaErrorInvalidConfiguration;
            }
            set.first[set.count] = int(p);
            const int grid = int(p < 1 ? 1 : min64(p, kBlocks));
            if (pass == 0) {
                clip_sum_kernel<<<grid, 256, 0, s>>>(set, part + nparts);
                nparts += grid;
            } else {
                clip_scale_kernel<<<grid, 256, 0, s>>>(set, part, nparts, max_norm, norm, l == 0);
            }
            const cudaError_t e = cudaGetLastError();
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace mgs
