// ds_cache.cu -- writing keys and values into a paged cache of 4-bit codes (ds_cache_store)
// and reading them back (ds_cache_load).
//
// A row (one token's key or value of one head, D numbers x) is held as D codes c in 0..15 and
// a bf16 pair (s, m), standing for s * c + m:
//   m = bf16(min x),  s = bf16((max x - m) / 15),  c = clamp(rint((x - m) / s), 0, 15).
// m and s are rounded before the codes are computed, so the codes make up for their rounding.
// Numbers up to 2^126 in size keep max - m and 15 s within fp32; beyond that s, or the value on
// loading, may be infinite.  A row whose s is below 2^-126 has codes 0 and stands for m: a constant
// row, and an fp32 row so narrow that m was rounded up past its maximum, whose s is negative.
//
// Layout: cache [pages][heads][page][2][D/2] bytes, key then value of a token side by side (at
// D = 128 one 128-byte line, so attention over scattered positions reads whole lines), two
// codes a byte, the even number in the low half; scales [pages][heads][page][4] bf16: key s,
// key m, value s, value m.  Token slot t is place t % page of page t / page.
//
// Both kernels move each byte once.  A token's key and value row of one head are neighbours in a
// warp.  Heads are the grid's second extent: no index is divided.
//
// Storing is bound by instructions (unpacking, the row's extremes, rounding), and what a row costs
// whatever its lanes (its places, its scale and their division, the exchanges) counts most: 32
// numbers a lane in pieces of 8.  16411 tokens of 8 heads in bf16: 15.4 us (5.5 TB/s); with 16
// numbers a lane 18.6, twice those with their loads in flight at once 20.7 (more registers, fewer
// warps to compute meanwhile), 64 numbers 15.4 and slower at 4096 tokens (5.1 us for 4.15).
// From fp32 23.4 us (6.5 TB/s).
//
// Loading is bound by its stores: a lane's piece is 16 bytes of numbers, so that a row's lanes write
// whole sectors side by side (fp32 by pairs of pieces: 37 us for 25), and its words of codes are
// 32 or 16 bits.  The same tokens: 12.3 us (6.9 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kCacheThreads = 128;
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
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store16(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

// Where a lane of LPR to a row works: `which` row (key 0, value 1), its lane of the row, and the
// token of turn k of U.
template <int LPR, int U>
struct Place {
    static constexpr int TPW = 16 / LPR, WARPS = kCacheThreads / 32;  // TPW: tokens per warp and turn
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

template <typename T, int D>
__global__ void __launch_bounds__(kCacheThreads) ds_cache_store_kernel(const CacheParams p) {
    constexpr int N = 4, LPR = D / (8 * N);  // N pieces of 8 numbers a lane
    pdl_launch_dependents();
    pdl_wait();
    const Place<LPR, 1> at;
    const int head = blockIdx.y;
    const int64_t token = at.token(0);
    const T* src = static_cast<const T*>(at.which ? p.v : p.k) + head * (at.which ? p.v_head : p.k_head) +
                   token * (at.which ? p.v_token : p.k_token) + at.sub * 8;
    float x[N][8];
    int64_t slot = -1;
    if (token < p.tokens) {
        slot = p.slots[token];
#pragma unroll
        for (int h = 0; h < N; ++h) load8<T>(src + h * (D / N), x[h]);
    } else {
#pragma unroll
        for (int i = 0; i < 8 * N; ++i) x[i / 8][i % 8] = 0.f;
    }
    float lo = fminf(x[0][0], x[0][1]), hi = fmaxf(x[0][0], x[0][1]);
#pragma unroll
    for (int i = 2; i < 8 * N; i += 2) {
        lo = min3(lo, x[i / 8][i % 8], x[i / 8][i % 8 + 1]);
        hi = max3(hi, x[i / 8][i % 8], x[i / 8][i % 8 + 1]);
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
    uint32_t word[N];
#pragma unroll
    for (int h = 0; h < N; ++h) {
        word[h] = 0u - kWhole * 0x11111111u;
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const float2 c = add_mul2(make_float2(x[h][i], x[h][i + 1]), -m, inv);
            word[h] += __float_as_uint(fmaxf(c.x, 0.f) + 8388608.f) << (4 * i);
            word[h] += __float_as_uint(fmaxf(c.y, 0.f) + 8388608.f) << (4 * i + 4);
        }
    }
    const int64_t entry = entry_of_slot(p, slot, head);
    if (entry < 0) return;
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.cache + entry * D + at.which * (D / 2)) + at.sub;
#pragma unroll
    for (int h = 0; h < N; ++h) dst[h * LPR] = word[h];
    if (at.sub == 0) p.scales[entry * 2 + at.which] = sb | mb << 16;
}

template <typename T, int D, int U>
__global__ void __launch_bounds__(kCacheThreads) ds_cache_load_kernel(const CacheParams p) {
    using Word = std::conditional_t<sizeof(T) == 2, uint32_t, uint16_t>;  // the codes of a piece
    constexpr int LPR = D / 16, PER = 16 / sizeof(T), N = 16 / PER;         // N pieces of PER numbers a lane
    pdl_launch_dependents();
    pdl_wait();
    const Place<LPR, U> at;
    const int head = blockIdx.y;
    uint32_t word[U][N], sm[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t token = at.token(k);
        const int64_t entry = token < p.tokens ? entry_of_slot(p, p.slots[token], head) : -1;
        sm[k] = 0u;  // a slot outside the cache: zeros
#pragma unroll
        for (int h = 0; h < N; ++h) word[k][h] = 0u;
        if (entry >= 0) {
            const Word* src = reinterpret_cast<const Word*>(p.cache + entry * D + at.which * (D / 2)) + at.sub;
#pragma unroll
            for (int h = 0; h < N; ++h) word[k][h] = src[h * LPR];
            sm[k] = p.scales[entry * 2 + at.which];
        }
    }
    T* dst = static_cast<T*>(const_cast<void*>(at.which ? p.v : p.k)) + head * (at.which ? p.v_head : p.k_head) + at.sub * PER;
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
        for (int h = 0; h < N; ++h) {
            float x[PER];
#pragma unroll
            for (int q = 0; q < PER / 4; ++q) {
                const uint32_t w = word[k][h] >> (16 * q);
                const float2 a = less_mul_add2(make_float2(__uint_as_float((w & 0xFu) | kWhole), __uint_as_float((w & 0xF0u) | kWhole)),
                                               8388608.f, s01, m);
                const float2 b = less_mul_add2(make_float2(__uint_as_float((w & 0xF00u) | kWhole), __uint_as_float((w & 0xF000u) | kWhole)),
                                               8388608.f, s23, m);
                x[4 * q] = a.x, x[4 * q + 1] = a.y, x[4 * q + 2] = b.x, x[4 * q + 3] = b.y;
            }
            store16(dst + token * stride + h * (D / N), x);
        }
    }
}

template <int LPR, int U, typename Kernel>
static ds_status launch_cache(Kernel kern, const CacheParams& p, cudaStream_t stream) {
    constexpr int64_t per = kCacheThreads / (2 * LPR) * U;  // tokens of a CTA
    if (p.tokens > 0x7FFFFFFFLL * per) return DS_ERR_UNSUPPORTED;
    const int64_t ctas = (p.tokens + per - 1) / per;
    return launch_pdl(kern, dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(p.heads)), kCacheThreads, 0, 1, stream, p);
}

// Loading takes two turns with all their loads in flight at once (16411 tokens: 12.3 us, with one
// 18.0), but one while that gives an SM less than 8 CTAs, as latency counts then (64 tokens: 1.3 us,
// with two 1.6).
template <typename T, int D>
static ds_status launch_cache(const CacheParams& p, bool store, int sms, cudaStream_t stream) {
    if (store) return launch_cache<D / 32, 1>(ds_cache_store_kernel<T, D>, p, stream);
    constexpr int LPR = D / 16;
    const int64_t ctas = p.tokens * p.heads / (kCacheThreads / (2 * LPR));
    return ctas < 8 * static_cast<int64_t>(sms) ? launch_cache<LPR, 1>(ds_cache_load_kernel<T, D, 1>, p, stream)
                                                : launch_cache<LPR, 2>(ds_cache_load_kernel<T, D, 2>, p, stream);
}

static ds_status cache_call(bool store, const void* k, const void* v, int32_t dtype, int64_t tokens, int32_t heads,
                            int32_t D, int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head, void* cache,
                            void* scales, int64_t pages, int32_t page, const int32_t* slots, cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || tokens < 0 || heads < 1 || pages < 0 || page < 1)
        return DS_ERR_INVALID_ARG;
    if ((page & (page - 1)) != 0 || (D != 64 && D != 128) || heads > 65535 || pages > INT64_MAX / page / heads / D)
        return DS_ERR_UNSUPPORTED;
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
