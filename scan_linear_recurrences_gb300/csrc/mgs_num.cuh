// Loads and stores of the language-model operators' element types (fp32 and
// bf16) with fp32 arithmetic between them.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

namespace mgs {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float x) { return __float2bfloat16_rn(x); }

// bf16 is the upper half of an fp32 word: the first of a pair in the low half
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// four consecutive elements
__device__ __forceinline__ void load4(const float *p, float (&v)[4]) {
    const float4 x = *reinterpret_cast<const float4 *>(p);
    v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
}
__device__ __forceinline__ void load4(const bf16 *p, float (&v)[4]) {
    const uint2 x = *reinterpret_cast<const uint2 *>(p);
    v[0] = bf_lo(x.x), v[1] = bf_hi(x.x), v[2] = bf_lo(x.y), v[3] = bf_hi(x.y);
}
__device__ __forceinline__ void store4(float *p, const float (&v)[4]) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(bf16 *p, const float (&v)[4]) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
}

// 16 bytes: kVec elements
template <typename T>
constexpr int kVec = 16 / int(sizeof(T));
__device__ __forceinline__ void unpack(const uint4 &u, float (&v)[4]) {
    v[0] = __uint_as_float(u.x), v[1] = __uint_as_float(u.y), v[2] = __uint_as_float(u.z), v[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(const uint4 &u, float (&v)[8]) {
    v[0] = bf_lo(u.x), v[1] = bf_hi(u.x), v[2] = bf_lo(u.y), v[3] = bf_hi(u.y);
    v[4] = bf_lo(u.z), v[5] = bf_hi(u.z), v[6] = bf_lo(u.w), v[7] = bf_hi(u.w);
}
__device__ __forceinline__ uint4 pack(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack(const float (&v)[8]) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// Two fp32 in a register pair, with sm_100's sums and products of pairs
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
__device__ __forceinline__ f2 pair(float x) { return pair(x, x); }

// (h, l) += (a, b), both sums of two fp32
__device__ __forceinline__ void add2(float &h, float &l, float a, float b) {
    const float s = h + a, t = s - h;
    const float e = (h - (s - t)) + (a - t);
    const float lo = l + b + e;
    h = s + lo;
    l = lo - (h - s);
}

// e^x as a sum of two fp32 (relative error about 1e-8), for factors that are
// multiplied together hundreds of times: x = n log 2 + y with |y| <= log(2) / 2
// (log 2 as 11357 / 2^14 and the rest, so that n times the first is exact: Cody
// and Waite's reduction), e^y = 1 + y + (Taylor's series from y^2 / 2), y and the
// sum in two parts.
__device__ __forceinline__ void exp_two(float x, float &hi, float &lo) {
    if (!(x > -100.f && x < 80.f)) {  // zero, overflow, NaN: nothing to refine
        hi = expf(x), lo = 0.f;
        return;
    }
    const float LN2_HI = 11357.f / 16384.f, LN2_LO = -2.9088971304690582e-5f;
    const float n = rintf(x * 1.44269504f);
    const float a = fmaf(-n, LN2_HI, x);  // exact
    const float b = -n * LN2_LO;
    const float y = a + b, yl = b - (y - a);
    float p = 1.f / 40320.f;
    p = fmaf(p, y, 1.f / 5040.f);
    p = fmaf(p, y, 1.f / 720.f);
    p = fmaf(p, y, 1.f / 120.f);
    p = fmaf(p, y, 1.f / 24.f);
    p = fmaf(p, y, 1.f / 6.f);
    p = fmaf(p, y, 0.5f);
    const float q = fmaf(p * y, y, yl + yl * y);
    const float s = 1.f + y, t = (1.f - s) + y;
    const float r = t + q;
    const float h = s + r, l = r - (h - s);
    const float e = ldexpf(1.f, int(n));
    hi = h * e, lo = l * e;
}

}  // namespace mgs
