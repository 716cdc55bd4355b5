// ds_cache.cu -- writing keys and values into a paged cache of 4-bit codes (ds_cache_store)
// and reading them back (ds_cache_load).
//
// A row (one token's key or value of one head, D numbers x) is held as D codes c in 0..15 and
// a bf16 pair (s, m), standing for s * c + m:
//   m = bf16(min x),  s = bf16((max x - m) / 15),  c = clamp(rint((x - m) / s), 0, 15).
// m and s are rounded before the codes are computed, so the codes make up for their rounding;
// bf16 has fp32's range, so no input of the supported types overflows them.  A row whose s is
// below 2^-126 (a constant row) has codes 0.
//
// Layout: cache [pages][heads][page][2][D/2] bytes, key then value of a token side by side (at
// D = 128 one 128-byte line, so attention over scattered positions reads whole lines), two
// codes a byte, the even number in the low half; scales [pages][heads][page][4] bf16: key s,
// key m, value s, value m.  Token slot t is place t % page of page t / page.
//
// Both kernels move each byte once.  A token's key and value row of one head are neighbours in a
// warp, D/16 lanes each, 16 numbers a lane (two pieces of 8: 16 bytes of bf16 in, 4 bytes of codes
// out), so a warp's code stores and loads are whole lines.  A warp takes U turns with all their
// loads in flight at once.  Heads are the grid's second extent: no index is divided.
// 16411 tokens of 8 heads in bf16, stored and read back: 36.7 us (4.6 TB/s); with 8 numbers a lane and plain
// conversions 50 us, bound by instructions (22 a number); one turn at a time 57 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kCacheThreads = 256;
constexpr uint32_t kWhole = 0x4B000000u;  // 2^23 as fp32: its low bits count ones

struct CacheParams {
    const void* k;        // store: inputs; load: outputs (written through)
    const void* v;
    int64_t k_token, k_head, v_token, v_head;  // element strides
    uint8_t* cache;
    uint32_t* scales;     // (s, m) pairs
    const int32_t* slots;
    int64_t tokens;
    int32_t heads, page_log;
    int64_t max_slot;     // pages * page
};

__device__ __forceinline__ uint32_t bf16_bits(float v) {
    return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v)));
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float low_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&x)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&x)[8]) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = low_bf16(w[i]);
        x[2 * i + 1] = high_bf16(w[i]);
    }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 q = reinterpret_cast<const float4*>(p)[i];
        x[4 * i] = q.x, x[4 * i + 1] = q.y, x[4 * i + 2] = q.z, x[4 * i + 3] = q.w;
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Where a lane works: `which` row (key 0, value 1), its lane of the row, and the token of turn k.
template <int D, int U>
struct Place {
    static constexpr int LPR = D / 16, TPW = 16 / LPR, WARPS = kCacheThreads / 32;  // tokens per warp and turn
    int which, sub;
    int64_t first;
    __device__ __forceinline__ Place() {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        which = lane / LPR & 1;
        sub = lane % LPR;
        first = static_cast<int64_t>(blockIdx.x) * (WARPS * TPW * U) + warp * TPW + lane / (2 * LPR);
    }
    __device__ __forceinline__ int64_t token(int k) const { return first + k * (WARPS * TPW); }
};

// two numbers to an instruction: (x + add) * by, and x * by + add
__device__ __forceinline__ float2 add_mul2(float2 x, float add, float by) {
    float2 r;
    asm("{\n\t.reg .b64 x, a, b;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 a, {%4, %4};\n\tmov.b64 b, {%5, %5};\n\t"
        "add.rn.f32x2 x, x, a;\n\tmul.rn.f32x2 x, x, b;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(add), "f"(by));
    return r;
}
__device__ __forceinline__ float2 less_mul_add2(float2 x, float less, float2 by, float add) {  // (x - less) * by + add
    float2 r;
    asm("{\n\t.reg .b64 x, l, b, a;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 l, {%4, %4};\n\tmov.b64 b, {%5, %6};\n\tmov.b64 a, {%7, %7};\n\t"
        "add.rn.f32x2 x, x, l;\n\tfma.rn.f32x2 x, x, b, a;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(-less), "f"(by.x), "f"(by.y), "f"(add));
    return r;
}

// The entry of a slot, or -1 for a slot outside the cache.
__device__ __forceinline__ int64_t entry_of_slot(const CacheParams& p, int64_t slot, int head) {
    if (slot < 0 || slot >= p.max_slot) return -1;
    const int64_t page = slot >> p.page_log, place = slot & ((int64_t(1) << p.page_log) - 1);
    return ((page * p.heads + head) << p.page_log) + place;
}

template <typename T, int D, int U>
__global__ void __launch_bounds__(kCacheThreads) ds_cache_store_kernel(const CacheParams p) {
    constexpr int LPR = D / 16;
    pdl_launch_dependents();
    pdl_wait();
    const Place<D, U> at;
    const int head = blockIdx.y;
    const T* src = static_cast<const T*>(at.which ? p.v : p.k) + head * (at.which ? p.v_head : p.k_head) + at.sub * 8;
    const int64_t stride = at.which ? p.v_token : p.k_token;
    float x[U][2][8];
    int64_t slot[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t token = at.token(k);
        slot[k] = -1;
        if (token < p.tokens) {
            slot[k] = p.slots[token];
            load8<T>(src + token * stride, x[k][0]);
            load8<T>(src + token * stride + D / 2, x[k][1]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[k][0][i] = x[k][1][i] = 0.f;
        }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        float lo = fminf(x[k][0][0], x[k][1][0]), hi = fmaxf(x[k][0][0], x[k][1][0]);
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            lo = min3(lo, x[k][0][i], x[k][1][i]);
            hi = max3(hi, x[k][0][i], x[k][1][i]);
        }
#pragma unroll
        for (int d = LPR / 2; d >= 1; d >>= 1) {
            lo = fminf(lo, __shfl_xor_sync(0xFFFFFFFFu, lo, d));
            hi = fmaxf(hi, __shfl_xor_sync(0xFFFFFFFFu, hi, d));
        }
        const uint32_t mb = bf16_bits(lo);
        const float m = low_bf16(mb);
        const uint32_t sb = bf16_bits((hi - m) * (1.0f / 15.0f));
        const float s = low_bf16(sb);
        const float inv = s >= 1.17549435e-38f ? 1.0f / s : 0.f;
        // Adding 2^23 rounds 0 .. 15 to a whole number, ties to even, and leaves it in the low bits;
        // the sum of the shifted words carries eight copies of 2^23's pattern, taken off beforehand.
        // (x - m) / s is at most 15 (1 + 2^-9) / (1 - 2^-9), which rounds to 15; it falls below 0
        // where m was rounded up.
        uint32_t word[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            word[h] = 0u - kWhole * 0x11111111u;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 c = add_mul2(make_float2(x[k][h][i], x[k][h][i + 1]), -m, inv);
                word[h] += __float_as_uint(fmaxf(c.x, 0.f) + 8388608.f) << (4 * i);
                word[h] += __float_as_uint(fmaxf(c.y, 0.f) + 8388608.f) << (4 * i + 4);
            }
        }
        const int64_t entry = entry_of_slot(p, slot[k], head);
        if (entry < 0) continue;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.cache + entry * D + at.which * (D / 2)) + at.sub;
        dst[0] = word[0];
        dst[LPR] = word[1];
        if (at.sub == 0) p.scales[entry * 2 + at.which] = sb | mb << 16;
    }
}

template <typename T, int D, int U>
__global__ void __launch_bounds__(kCacheThreads) ds_cache_load_kernel(const CacheParams p) {
    constexpr int LPR = D / 16;
    pdl_launch_dependents();
    pdl_wait();
    const Place<D, U> at;
    const int head = blockIdx.y;
    uint32_t word[U][2], sm[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t token = at.token(k);
        const int64_t entry = token < p.tokens ? entry_of_slot(p, p.slots[token], head) : -1;
        word[k][0] = word[k][1] = sm[k] = 0u;  // a slot outside the cache: zeros
        if (entry >= 0) {
            const uint32_t* src = reinterpret_cast<const uint32_t*>(p.cache + entry * D + at.which * (D / 2)) + at.sub;
            word[k][0] = src[0];
            word[k][1] = src[LPR];
            sm[k] = p.scales[entry * 2 + at.which];
        }
    }
    T* dst = static_cast<T*>(const_cast<void*>(at.which ? p.v : p.k)) + head * (at.which ? p.v_head : p.k_head) + at.sub * 8;
    const int64_t stride = at.which ? p.v_token : p.k_token;
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t token = at.token(k);
        if (token >= p.tokens) continue;
        // A code in place, under 2^23's pattern, is 2^23 + c 16^i; s c is exact in fp32 (8 by 4 bits),
        // so m is added with one rounding.
        const float s = low_bf16(sm[k]), m = high_bf16(sm[k]);
        const float2 s01 = make_float2(s, s * 0.0625f), s23 = make_float2(s * 0.00390625f, s * 0.000244140625f);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float x[8];
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                const uint32_t w = word[k][h] >> (16 * q);
                const float2 a = less_mul_add2(make_float2(__uint_as_float((w & 0xFu) | kWhole), __uint_as_float((w & 0xF0u) | kWhole)),
                                               8388608.f, s01, m);
                const float2 b = less_mul_add2(make_float2(__uint_as_float((w & 0xF00u) | kWhole), __uint_as_float((w & 0xF000u) | kWhole)),
                                               8388608.f, s23, m);
                x[4 * q] = a.x, x[4 * q + 1] = a.y, x[4 * q + 2] = b.x, x[4 * q + 3] = b.y;
            }
            store8(dst + token * stride + h * (D / 2), x);
        }
    }
}

template <typename T, int D, int U>
static ds_status launch_cache(const CacheParams& p, bool store, cudaStream_t stream) {
    constexpr int64_t per = kCacheThreads / (D / 8) * U;  // tokens of a CTA
    const int64_t ctas = (p.tokens + per - 1) / per;
    if (ctas > 0x7FFFFFFFLL) return DS_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(ctas), static_cast<unsigned>(p.heads));
    return store ? launch_pdl(ds_cache_store_kernel<T, D, U>, grid, kCacheThreads, 0, 1, stream, p)
                 : launch_pdl(ds_cache_load_kernel<T, D, U>, grid, kCacheThreads, 0, 1, stream, p);
}

// One turn while that gives an SM less than 8 CTAs (latency counts), else two.
template <typename T, int D>
static ds_status launch_cache(const CacheParams& p, bool store, int sms, cudaStream_t stream) {
    const int64_t ctas = p.tokens * p.heads / (kCacheThreads / (D / 8));
    return ctas < 8 * static_cast<int64_t>(sms) ? launch_cache<T, D, 1>(p, store, stream) : launch_cache<T, D, 2>(p, store, stream);
}

static ds_status cache_call(bool store, const void* k, const void* v, int32_t dtype, int64_t tokens, int32_t heads,
                            int32_t D, int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head, void* cache,
                            void* scales, int64_t pages, int32_t page, const int32_t* slots, cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || tokens < 0 || heads < 1 || pages < 0 || page < 1)
        return DS_ERR_INVALID_ARG;
    if ((page & (page - 1)) != 0 || (D != 64 && D != 128) || heads > 65535) return DS_ERR_UNSUPPORTED;
    if (k_token < 0 || k_head < 0 || v_token < 0 || v_head < 0) return DS_ERR_INVALID_ARG;
    if (tokens == 0) return DS_OK;
    if (!k || !v || !slots || (pages > 0 && (!cache || !scales))) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    const int64_t strides[] = {k_token, k_head, v_token, v_head};
    for (int64_t s : strides)
        if (s * es % 16) return DS_ERR_ALIGNMENT;
    if (!aligned16(k) || !aligned16(v) || !aligned16(cache) || reinterpret_cast<uintptr_t>(scales) % 8 ||
        reinterpret_cast<uintptr_t>(slots) % 4)
        return DS_ERR_ALIGNMENT;
    CacheParams p = {};
    p.k = k;
    p.v = v;
    p.k_token = k_token;
    p.k_head = k_head;
    p.v_token = v_token;
    p.v_head = v_head;
    p.cache = static_cast<uint8_t*>(cache);
    p.scales = static_cast<uint32_t*>(scales);
    p.slots = slots;
    p.tokens = tokens;
    p.heads = heads;
    while ((1 << p.page_log) < page) ++p.page_log;
    p.max_slot = pages * page;
    int dev = 0;
    DevInfo info;
    if (cudaGetDevice(&dev) != cudaSuccess || !dev_info(dev, info)) return DS_ERR_CUDA;
    if (dtype == DS_BF16)
        return D == 64 ? launch_cache<__nv_bfloat16, 64>(p, store, info.sms, stream)
                       : launch_cache<__nv_bfloat16, 128>(p, store, info.sms, stream);
    return D == 64 ? launch_cache<float, 64>(p, store, info.sms, stream) : launch_cache<float, 128>(p, store, info.sms, stream);
}

}  // namespace dsk

using namespace dsk;

extern "C" {

ds_status ds_cache_store(const void* k, const void* v, int32_t dtype, int64_t tokens, int32_t heads, int32_t D,
                         int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride,
                         void* cache, void* scales, int64_t pages, int32_t page, const int32_t* slots,
                         cudaStream_t stream) {
    return cache_call(true, k, v, dtype, tokens, heads, D, k_token_stride, k_head_stride, v_token_stride, v_head_stride,
                      cache, scales, pages, page, slots, stream);
}

ds_status ds_cache_load(const void* cache, const void* scales, int64_t pages, int32_t page, const int32_t* slots,
                        int64_t tokens, int32_t heads, int32_t D, int32_t dtype, void* out_k, void* out_v,
                        cudaStream_t stream) {
    const int64_t row = D, token = static_cast<int64_t>(heads) * D;
    return cache_call(false, out_k, out_v, dtype, tokens, heads, D, token, row, token, row, const_cast<void*>(cache),
                      const_cast<void*>(scales), pages, page, slots, stream);
}

}  // extern "C"
