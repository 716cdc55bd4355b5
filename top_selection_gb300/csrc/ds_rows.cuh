// ds_rows.cuh -- device helpers of the kernels that stream rows: 16 bytes of a row as fp32 and
// back, sums over lanes, and the 8-bit form of numbers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ds_common.cuh"

namespace dsk {

// bf16 is the upper half of fp32's bits.
__device__ __forceinline__ float row_f32(float v) { return v; }
__device__ __forceinline__ float row_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void row_put(float* p, float v) { *p = v; }
__device__ __forceinline__ void row_put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

template <typename T>
constexpr int kPer = 16 / static_cast<int>(sizeof(T));  // numbers in 16 bytes

__device__ __forceinline__ void unpack16(const uint4& q, float (&v)[4]) {
    v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void unpack16(const uint4& q, float (&v)[8]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack16(const float (&v)[4]) {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ uint4 pack16(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Sum over runs of N lanes, the same in every lane.
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int d = N / 2; d >= 1; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}
template <int N>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int d = N / 2; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

// The scale of an 8-bit block whose largest number is `top`: the least power of two s >= 2^-126 with
// top <= 448 s.  448 is 1.75 * 2^8: the exponent of top less 8, one more where its fraction is above
// 1.75 (adding 2^21 - 1 to the bits carries into the exponent just there).
__device__ __forceinline__ float block_scale(float top) {
    const int field = static_cast<int>((__float_as_uint(top) + 0x1FFFFFu) >> 23) - 8;
    return __uint_as_float(static_cast<uint32_t>(field < 1 ? 1 : field) << 23);
}
// 1 / s of such a scale: its exponent negated, exactly.
__device__ __forceinline__ float block_inverse(float s) { return __uint_as_float(0x7F000000u - __float_as_uint(s)); }

// Two numbers as e4m3, rounded to nearest, ties to even; the first in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t e4m3_four(float a, float b, float c, float d) {
    return e4m3_pair(a, b) | e4m3_pair(c, d) << 16;
}

}  // namespace dsk
