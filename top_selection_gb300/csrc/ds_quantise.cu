// ds_quantise.cu -- rows and weights in 8 bits with a scale for each block of 128
// (ds_quantise_blocks), and the experts' gather that gives its rows in that form
// (ds_expert_gather_quantised).
//
// A block of numbers (128 of a row, or 128 x 128 of a matrix) has the scale s, the least power of
// two that brings its largest number to e4m3's 448 or below, and codes e4m3(x / s).  The division by
// a power of two is exact, so a code is x / s rounded once: half a step, 2^-4 of the number (or
// 2^-10 s below 2^-6 s).  Infinities and NaN have the code NaN; for its block's scale an infinity counts like the largest
// number, a NaN not at all.  Bound by memory: 16411 x 2048 bf16 in 14.4 us (7.1 TB/s), 16 x 2000 x 4096 fp32 in
// blocks of 128 x 128 in 95.2 (6.9), bf16 in 57.0.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_rows.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kQuantThreads = 256;
constexpr int kQuantMaxE = 512, kQuantMaxK = 32;
constexpr int kQuantMaxColumns = 1 << 26;  // 32768 runs of 16 blocks (a grid has 65535); columns are counted in 32 bits

constexpr float kMostScale = 1329227995784915872903807060280344576.f;  // 2^120, of a block that holds an infinity

struct QuantParams {
    const void* x;
    uint8_t* codes;
    float* scales;
    int64_t matrices, rows, matrix_stride, stride;  // rows of each matrix
    int32_t K, blocks;                              // numbers of a row, blocks of 128 in it
    int32_t side;                                   // log2 of the blocks of a row that a CTA takes at a time
    // the gather: k places of each row, and the rows behind the last place
    const int32_t* places;
    const int32_t* offsets;
    int32_t k, E;
};

// A lane's 16 numbers of a row's 128, 8 lanes to them: two runs of 8, 64 apart (VEC), or every 8th one.  Sizes of bf16
// numbers are compared two at a time, and half as many lanes share the work on a scale as with 8 numbers
// each (16411 x 2048 bf16: 25.3 us then, 14.3 now; fp32 25.3 and 25.5, its bytes).
template <typename T, bool VEC>
struct Sixteen {
    static constexpr int WORDS = static_cast<int>(sizeof(T));  // of 16 bytes
    uint4 q[WORDS];
    float v[16];
    __device__ __forceinline__ void load(const T* row, int first, int K, int sub) {
        if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const int at = first + sub * 8 + 64 * (i / (WORDS / 2)) + kPer<T> * (i % (WORDS / 2));
                q[i] = at < K ? *reinterpret_cast<const uint4*>(row + at) : make_uint4(0u, 0u, 0u, 0u);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int at = first + sub + 8 * j;
                v[j] = at < K ? row_f32(row[at]) : 0.f;
            }
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) q[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.f;
    }
    __device__ __forceinline__ float most() const {  // the largest size among them, NaN left out
        if constexpr (VEC && sizeof(T) == 2) {  // two bf16 numbers at a time, signs cleared
            const auto pair = [](uint32_t u) {
                u &= 0x7FFF7FFFu;
                return *reinterpret_cast<const __nv_bfloat162*>(&u);
            };
            const auto word = [&](const uint4& w) { return __hmax2(__hmax2(pair(w.x), pair(w.y)), __hmax2(pair(w.z), pair(w.w))); };
            const __nv_bfloat162 m = __hmax2(word(q[0]), word(q[1]));
            return fmaxf(fmaxf(__low2float(m), __high2float(m)), 0.f);
        } else {
            float m = 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) m = fmaxf(m, fabsf(number(j)));
            return m;
        }
    }
    __device__ __forceinline__ float number(int j) const {
        if constexpr (!VEC) {
            return v[j];
        } else {
            constexpr int PER = kPer<T>;
            float f[PER];
            unpack16(q[j / PER], f);
            return f[j % PER];
        }
    }
    // Codes of numbers in a block of scale s.  The conversion saturates, and no code stands for an infinity: at
    // s = 2^120 finite numbers are 2^8 at most, so that 448 (0x7E) there is an infinity, and becomes NaN (0x7F): a few
    // instructions for four numbers, where a select before the conversion takes two for each.
    __device__ __forceinline__ uint4 codes(float s) const {
        const float inv = block_inverse(s);
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            c[i] = e4m3_four(number(4 * i) * inv, number(4 * i + 1) * inv, number(4 * i + 2) * inv, number(4 * i + 3) * inv);
        if (s == kMostScale) {
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] |= (((c[i] & 0x7F7F7F7Fu) + 0x02020202u) >> 7) & 0x01010101u;
        }
        return make_uint4(c[0], c[1], c[2], c[3]);
    }
};
template <bool VEC>
__device__ __forceinline__ void store_sixteen(uint8_t* row, int first, int K, int sub, uint4 c) {
    if constexpr (VEC) {
        const int at = first + sub * 8;
        if (at < K) *reinterpret_cast<uint2*>(row + at) = make_uint2(c.x, c.y);
        if (at + 64 < K) *reinterpret_cast<uint2*>(row + at + 64) = make_uint2(c.z, c.w);
    } else {
        const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int at = first + sub + 8 * j;
            if (at < K) row[at] = static_cast<uint8_t>(w[j / 4] >> (8 * (j & 3)));
        }
    }
}

// Blocks of rows: 8 lanes to a block, 32 blocks to a CTA at a time, 2^side of them of one row (`side` is 4 where
// rows have more than 8 blocks); kQuantUnits rows to a lane, all loaded before the first is used.
// blockIdx.y counts the runs of 2^side blocks of a row.
constexpr int kQuantUnits = 2;
constexpr int kQuantLog = 5;  // log2 of the blocks to a CTA at a time

template <typename T, bool VEC, bool GATHER>
__global__ void __launch_bounds__(kQuantThreads) ds_quantise_rows_kernel(const QuantParams p) {
    const int sub = threadIdx.x & 7, team = threadIdx.x >> 3;
    pdl_launch_dependents();
    pdl_wait();
    constexpr int UNITS = GATHER ? 1 : kQuantUnits;
    const int64_t all_rows = p.matrices * p.rows;
    const int down = kQuantLog - p.side;  // log2 of the rows at a time
    const int64_t row0 = (static_cast<int64_t>(blockIdx.x) * UNITS << down) + (team >> p.side);
    const int block = static_cast<int>(blockIdx.y << p.side) + (team & ((1 << p.side) - 1));
    Sixteen<T, VEC> v[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int64_t r = min(row0 + (i << down), all_rows - 1);
        const int64_t m = p.matrices == 1 ? 0 : r / p.rows;
        v[i].load(static_cast<const T*>(p.x) + m * p.matrix_stride + (r - m * p.rows) * p.stride, block * 128, p.K, sub);
    }
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const float s = block_scale(lanes_max<8>(v[i].most()));
        const uint4 c = v[i].codes(s);
        if constexpr (!GATHER) {
            const int64_t row = row0 + (i << down);
            if (row >= all_rows || block >= p.blocks) continue;  // (the warp stays whole for its shuffles)
            store_sixteen<VEC>(p.codes + row * p.K, block * 128, p.K, sub, c);
            if (sub == 0) p.scales[row * p.blocks + block] = s;
        } else {
            if (row0 >= all_rows || block >= p.blocks) return;
            const int64_t slots = p.rows * p.k, first = row0 * p.k;
            for (int j = 0; j < p.k; ++j) {
                const int64_t at = p.places[first + j];
                if (at < 0 || at >= slots) continue;
                store_sixteen<VEC>(p.codes + at * p.K, block * 128, p.K, sub, c);
                if (sub == 0) p.scales[at * p.blocks + block] = s;
            }
            const int64_t filled = p.offsets[p.E];
            for (int64_t at = max(filled, first); at < first + p.k; ++at) {  // a row of zeros
                store_sixteen<VEC>(p.codes + at * p.K, block * 128, p.K, sub, make_uint4(0u, 0u, 0u, 0u));
                if (sub == 0) p.scales[at * p.blocks + block] = block_scale(0.f);
            }
        }
    }
}

// Blocks of 128 x 128: a CTA holds one in registers, 8 lanes to a row, 4 rows to a lane.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kQuantThreads) ds_quantise_tiles_kernel(const QuantParams p) {
    constexpr int TEAMS = kQuantThreads / 8, R = 128 / TEAMS;
    __shared__ float sh_max[kQuantThreads / 32];
    const int sub = threadIdx.x & 7, team = threadIdx.x >> 3;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t tall = (p.rows + 127) / 128;
    const int64_t strip = blockIdx.x / p.blocks, m = strip / tall;
    const int block = static_cast<int>(blockIdx.x - strip * p.blocks);
    const int64_t row0 = (strip - m * tall) * 128;
    const T* x = static_cast<const T*>(p.x) + m * p.matrix_stride;
    Sixteen<T, VEC> v[R];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t r = row0 + team + i * TEAMS;
        if (r < p.rows) v[i].load(x + r * p.stride, block * 128, p.K, sub);
        else v[i].clear();
    }
#pragma unroll
    for (int i = 0; i < R; ++i) top = fmaxf(top, v[i].most());
    top = lanes_max<32>(top);
    if (threadIdx.x % 32 == 0) sh_max[threadIdx.x / 32] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuantThreads / 32; ++w) top = fmaxf(top, sh_max[w]);
    const float s = block_scale(top);
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t r = row0 + team + i * TEAMS;
        if (r < p.rows) store_sixteen<VEC>(p.codes + (m * p.rows + r) * p.K, block * 128, p.K, sub, v[i].codes(s));
    }
    if (threadIdx.x == 0) p.scales[blockIdx.x] = s;
}

// ---------------------------------------------------------------- host --------------
template <typename T>
static ds_status launch_quantise(QuantParams p, int block_rows, bool vec, bool gather, cudaStream_t stream) {
    const auto go = [&](auto kern, int64_t ctas, int64_t runs) {
        if (ctas > 0x7FFFFFFFLL || runs > 65535) return DS_ERR_UNSUPPORTED;
        return launch_pdl(kern, dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(runs)), kQuantThreads, 0, 1, stream, p);
    };
    if (block_rows == 128) {
        const int64_t ctas = p.matrices * ((p.rows + 127) / 128) * p.blocks;
        return vec ? go(ds_quantise_tiles_kernel<T, true>, ctas, 1) : go(ds_quantise_tiles_kernel<T, false>, ctas, 1);
    }
    p.side = 0;
    while (p.side < 4 && (1 << p.side) < p.blocks) ++p.side;
    const int64_t at_once = (gather ? 1LL : kQuantUnits) << (kQuantLog - p.side), ctas = (p.matrices * p.rows + at_once - 1) / at_once;
    const int64_t runs = (p.blocks + (1LL << p.side) - 1) >> p.side;
    if (gather) return vec ? go(ds_quantise_rows_kernel<T, true, true>, ctas, runs) : go(ds_quantise_rows_kernel<T, false, true>, ctas, runs);
    return vec ? go(ds_quantise_rows_kernel<T, true, false>, ctas, runs) : go(ds_quantise_rows_kernel<T, false, false>, ctas, runs);
}

static bool not_on(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

}  // namespace dsk

using namespace dsk;

extern "C" {

ds_status ds_quantise_blocks(const void* x, int32_t dtype, int64_t matrices, int64_t rows, int32_t K,
                             int64_t matrix_stride, int64_t row_stride, int32_t block_rows, void* codes, float* scales,
                             cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || matrices < 0 || rows < 0 || K < 1 || row_stride < K || matrix_stride < 0 ||
        (block_rows != 1 && block_rows != 128))
        return DS_ERR_INVALID_ARG;
    if (K > kQuantMaxColumns) return DS_ERR_UNSUPPORTED;
    const int64_t limit = 1LL << 40;  // numbers in all, and their reach in x
    if (rows > limit / K || (rows > 0 && matrices > limit / K / rows) || (rows > 0 && row_stride > (limit << 8) / rows) ||
        (matrices > 0 && matrix_stride > (limit << 8) / matrices))
        return DS_ERR_UNSUPPORTED;
    if (matrices == 0 || rows == 0) return DS_OK;
    if (!x || !codes || !scales) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    if (not_on(x, es) || not_on(scales, 4)) return DS_ERR_ALIGNMENT;
    QuantParams p = {x, static_cast<uint8_t*>(codes), scales, matrices, rows, matrix_stride, row_stride, K, (K + 127) / 128, 0,
                     nullptr, nullptr, 0, 0};
    if (block_rows == 1 && (matrices == 1 || matrix_stride == rows * row_stride)) p.rows = matrices * rows, p.matrices = 1;
    const bool vec = K % 8 == 0 && aligned16(x) && !not_on(codes, 8) && row_stride * es % 16 == 0 &&
                     (matrices == 1 || matrix_stride * es % 16 == 0);
    return dtype == DS_BF16 ? launch_quantise<__nv_bfloat16>(p, block_rows, vec, false, stream)
                            : launch_quantise<float>(p, block_rows, vec, false, stream);
}

ds_status ds_expert_gather_quantised(const void* x, int32_t dtype, int64_t tokens, int32_t D, int64_t row_stride,
                                     const int32_t* places, int32_t k, const int32_t* offsets, int32_t E, void* codes,
                                     float* scales, cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || tokens < 0 || D < 1 || k < 1 || row_stride < D || E < 1)
        return DS_ERR_INVALID_ARG;
    if (k > kQuantMaxK || E > kQuantMaxE || D > kQuantMaxColumns || tokens > 0x7FFFFFFFLL / k) return DS_ERR_UNSUPPORTED;
    if (tokens == 0) return DS_OK;
    if (!x || !places || !offsets || !codes || !scales) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    if (not_on(x, es) || not_on(scales, 4) || not_on(places, 4) || not_on(offsets, 4)) return DS_ERR_ALIGNMENT;
    const QuantParams p = {x, static_cast<uint8_t*>(codes), scales, 1, tokens, 0, row_stride, D, (D + 127) / 128, 0,
                           places, offsets, k, E};
    const bool vec = D % 8 == 0 && aligned16(x) && !not_on(codes, 8) && row_stride * es % 16 == 0;
    return dtype == DS_BF16 ? launch_quantise<__nv_bfloat16>(p, 1, vec, true, stream)
                            : launch_quantise<float>(p, 1, vec, true, stream);
}

}  // extern "C"
