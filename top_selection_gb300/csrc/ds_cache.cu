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
// Both kernels move each byte once: D/8 lanes per row, 8 numbers a lane (16 bytes of bf16 in,
// 4 bytes of codes out); a token's key and value rows are neighbours in a warp, so a warp's
// code stores and loads are whole lines.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kCacheThreads = 256;

struct CacheParams {
    const void* k;        // store: inputs; load: outputs (written through)
    const void* v;
    int64_t k_token, k_head, v_token, v_head;  // element strides
    uint8_t* cache;
    uint32_t* scales;     // (s, m) pairs
    const int32_t* slots;
    int64_t units;        // tokens * heads * 2 rows
    int32_t heads, page_log;
    int64_t max_slot;     // pages * page
};

__device__ __forceinline__ uint32_t bf16_bits(float v) {
    return static_cast<uint32_t>(__bfloat16_as_ushort(__float2bfloat16_rn(v)));
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
    for (int i = 0; i < 4; ++i) w[i] = bf16_bits(x[2 * i]) | bf16_bits(x[2 * i + 1]) << 16;
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// Row u of the call: token, head, and key (0) or value (1); LPR lanes share it.
template <int LPR>
struct RowOf {
    int64_t unit, token;
    int lane, head, which;
    bool on;
    __device__ __forceinline__ RowOf(int64_t units, int heads) {
        const int64_t th = static_cast<int64_t>(blockIdx.x) * kCacheThreads + threadIdx.x;
        unit = th / LPR;
        lane = static_cast<int>(th % LPR);
        on = unit < units;
        which = static_cast<int>(unit & 1);
        token = (unit >> 1) / heads;
        head = static_cast<int>((unit >> 1) % heads);
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kCacheThreads) ds_cache_store_kernel(const CacheParams p) {
    constexpr int LPR = D / 8;
    pdl_launch_dependents();
    pdl_wait();
    const RowOf<LPR> r(p.units, p.heads);
    float x[8];
    int64_t slot = -1;
    if (r.on) {
        slot = p.slots[r.token];
        const T* src = static_cast<const T*>(r.which ? p.v : p.k) +
                       r.token * (r.which ? p.v_token : p.k_token) + r.head * (r.which ? p.v_head : p.k_head);
        load8<T>(src + r.lane * 8, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
    float lo = x[0], hi = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) lo = fminf(lo, x[i]), hi = fmaxf(hi, x[i]);
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
    uint32_t word = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = fminf(fmaxf(rintf((x[i] - m) * inv), 0.f), 15.f);
        word |= static_cast<uint32_t>(c) << (4 * i);
    }
    if (!r.on || slot < 0 || slot >= p.max_slot) return;
    const int64_t page = slot >> p.page_log, place = slot & ((int64_t(1) << p.page_log) - 1);
    const int64_t entry = ((page * p.heads + r.head) << p.page_log) + place;
    reinterpret_cast<uint32_t*>(p.cache + entry * D + r.which * (D / 2))[r.lane] = word;
    if (r.lane == 0) p.scales[entry * 2 + r.which] = sb | mb << 16;
}

template <typename T, int D>
__global__ void __launch_bounds__(kCacheThreads) ds_cache_load_kernel(const CacheParams p) {
    constexpr int LPR = D / 8;
    pdl_launch_dependents();
    pdl_wait();
    const RowOf<LPR> r(p.units, p.heads);
    if (!r.on) return;
    const int64_t slot = p.slots[r.token];
    float x[8];
    if (slot >= 0 && slot < p.max_slot) {
        const int64_t page = slot >> p.page_log, place = slot & ((int64_t(1) << p.page_log) - 1);
        const int64_t entry = ((page * p.heads + r.head) << p.page_log) + place;
        const uint32_t word = reinterpret_cast<const uint32_t*>(p.cache + entry * D + r.which * (D / 2))[r.lane];
        const uint32_t sm = p.scales[entry * 2 + r.which];
        // s * c is exact in fp32 (8 by 4 bits): one rounding, with or without a fused add
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = low_bf16(sm) * static_cast<float>((word >> (4 * i)) & 15u) + high_bf16(sm);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = 0.f;
    }
    T* dst = static_cast<T*>(const_cast<void*>(r.which ? p.v : p.k)) +
             r.token * (r.which ? p.v_token : p.k_token) + r.head * (r.which ? p.v_head : p.k_head);
    store8(dst + r.lane * 8, x);
}

static ds_status cache_call(bool store, const void* k, const void* v, int32_t dtype, int64_t tokens, int32_t heads,
                            int32_t D, int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head, void* cache,
                            void* scales, int64_t pages, int32_t page, const int32_t* slots, cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || tokens < 0 || heads < 1 || pages < 0 || page < 1)
        return DS_ERR_INVALID_ARG;
    if ((page & (page - 1)) != 0 || (D != 64 && D != 128)) return DS_ERR_UNSUPPORTED;
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
    p.units = tokens * heads * 2;
    p.heads = heads;
    while ((1 << p.page_log) < page) ++p.page_log;
    p.max_slot = pages * page;
    const int64_t ctas = (p.units * (D / 8) + kCacheThreads - 1) / kCacheThreads;
    if (ctas > 0x7FFFFFFFLL) return DS_ERR_UNSUPPORTED;
    const dim3 grid(static_cast<unsigned>(ctas));
    const auto go = [&](auto kern) { return launch_pdl(kern, grid, kCacheThreads, 0, 1, stream, p); };
    if (store) {
        if (dtype == DS_BF16)
            return D == 64 ? go(ds_cache_store_kernel<__nv_bfloat16, 64>) : go(ds_cache_store_kernel<__nv_bfloat16, 128>);
        return D == 64 ? go(ds_cache_store_kernel<float, 64>) : go(ds_cache_store_kernel<float, 128>);
    }
    if (dtype == DS_BF16)
        return D == 64 ? go(ds_cache_load_kernel<__nv_bfloat16, 64>) : go(ds_cache_load_kernel<__nv_bfloat16, 128>);
    return D == 64 ? go(ds_cache_load_kernel<float, 64>) : go(ds_cache_load_kernel<float, 128>);
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
