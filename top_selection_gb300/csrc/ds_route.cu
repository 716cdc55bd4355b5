// ds_route.cu -- the experts' gate: top-k of a short row of scores (ds_route), and the
// gradient of the weights it returns (ds_route_backward).
//
// A row x of E logits has scores s = softmax(x) or s = 1 / (1 + exp(-x)).  The choice value
// of expert e is c_e = s_e + bias_e; without a bias the experts are ordered by x itself,
// which orders s exactly (exp and the logistic function rise strictly; their roundings do
// not).  With g groups of E/g consecutive experts, a group's score is its largest c or the
// sum of its two largest, and only experts of the topk_groups best groups stay.  The k
// largest c are chosen; every tie goes to the lowest index.  Weights are
//   w_j = scale * s_j / (renormalise ? sum of the chosen s : 1).
//
// One warp per row, the row in registers: lane l holds n consecutive experts of one group
// (each group has a power-of-two number of lanes), so lanes ascend with the experts and the
// lowest lane holding a maximum holds the lowest expert.  Selection is k rounds of: largest
// key of the lane, largest of the warp (redux.sync on the order-preserving integer key),
// lowest lane that has it (ballot), and that lane drops its first copy.  Lane j < k keeps
// the j-th choice, reads its logit again (the row is in L1) and computes its weight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kRouteWarps = 8;     // rows per CTA
constexpr int kRouteMaxE = 512;
constexpr int kRouteMaxK = 32;     // one lane per choice
constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

__device__ __forceinline__ float warp_sum_f32(float v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}
__device__ __forceinline__ float warp_max_f32(float v) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
    return v;
}

// expf and an IEEE division, not their fast forms: the sum with the bias decides which
// expert is chosen, so the score is the same number that the definition in fp32 gives.
__device__ __forceinline__ float logistic(float x) { return 1.0f / (1.0f + expf(-x)); }

// A softmax row of -inf alone has scores of zero, not NaN: its largest logit counts as 0
// and the sum of its exponentials as 1.
__device__ __forceinline__ float row_max(float m) { return m == -INFINITY ? 0.f : m; }
__device__ __forceinline__ float row_sum(float s) { return s == 0.f ? 1.f : s; }

struct RouteParams {
    const void* logits;
    const float* bias;
    float* weights;
    int32_t* experts;
    int32_t* counts;
    int64_t rows, row_stride;
    int32_t E, k, groups, topk_groups;
    int32_t size;     // experts per group
    int32_t llog;     // log2 of the lanes per group
    int32_t n;        // experts per lane, ceil(size / lanes)
    int32_t sigmoid, top2, renormalise;
    float scale;
};

// Loads the lane's n experts (a run of the row) as fp32; places past the run keep `fill`.
// VEC: rows and runs start on 16 bytes and n fills whole 16-byte words.
template <typename T, int EPL, bool VEC>
__device__ __forceinline__ void load_run(const T* src, int count, float fill, float (&v)[EPL]) {
    if (VEC && count == EPL && EPL * sizeof(T) >= 16) {
        constexpr int PER = 16 / sizeof(T);
#pragma unroll
        for (int i = 0; i < EPL / PER; ++i) {
            const uint4 q = reinterpret_cast<const uint4*>(src)[i];
            const T* e = reinterpret_cast<const T*>(&q);
#pragma unroll
            for (int j = 0; j < PER; ++j) v[i * PER + j] = to_f32(e[j]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = i < count ? to_f32(src[i]) : fill;
}

template <typename T, int EPL, bool VEC>
__global__ void __launch_bounds__(kRouteWarps * 32) ds_route_kernel(const RouteParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    pdl_launch_dependents();
    pdl_wait();
    if (row >= p.rows) return;
    const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
    const int lanes = 1 << p.llog;
    const int grp = lane >> p.llog, pos = lane & (lanes - 1);
    int count = min(p.n, p.size - pos * p.n);
    if (grp >= p.groups || count < 0) count = 0;
    const int first = grp * p.size + pos * p.n;  // the lane's first expert (when count > 0)
    float v[EPL];
    load_run<T, EPL, VEC>(x + (count > 0 ? first : 0), count, -INFINITY, v);

    // softmax: the row's largest logit and the sum of exponentials
    float mx = 0.f, total = 1.f;
    if (!p.sigmoid) {
        float m = v[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) m = fmaxf(m, v[i]);
        mx = row_max(warp_max_f32(m));
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) s += i < count ? expf(v[i] - mx) : 0.f;
        total = row_sum(warp_sum_f32(s));
    }
    // choice values; places past the run get key 0, below every value's key
    uint32_t key[EPL];
    if (p.bias) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (i < count) {
                const float s = p.sigmoid ? logistic(v[i]) : expf(v[i] - mx) / total;
                v[i] = s + p.bias[first + i];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i)  // + 0.f: -0 and +0 are equal
        key[i] = i < count ? max(key_f32(__float_as_uint(v[i] + 0.f)), 1u) : 0u;

    if (p.groups > 1) {
        uint32_t score;
        if (!p.top2) {
            uint32_t m = key[0];
#pragma unroll
            for (int i = 1; i < EPL; ++i) m = max(m, key[i]);
            for (int d = lanes >> 1; d >= 1; d >>= 1) m = max(m, __shfl_xor_sync(kFull, m, d));
            score = m;
        } else {
            // the two largest, merged across the group's lanes; without a bias the scores
            // themselves are added (softmax: before the division by their common sum)
            float a = -INFINITY, b = -INFINITY;
#pragma unroll
            for (int i = 0; i < EPL; ++i) {
                if (i < count) {
                    const float t = p.bias ? v[i] : p.sigmoid ? logistic(v[i]) : expf(v[i] - mx);
                    b = fmaxf(b, fminf(a, t));
                    a = fmaxf(a, t);
                }
            }
            for (int d = lanes >> 1; d >= 1; d >>= 1) {
                const float a2 = __shfl_xor_sync(kFull, a, d), b2 = __shfl_xor_sync(kFull, b, d);
                b = fmaxf(fminf(a, a2), fmaxf(b, b2));
                a = fmaxf(a, a2);
            }
            score = key_f32(__float_as_uint((p.size > 1 ? a + b : a) + 0.f));
        }
        int rank = 0;
        for (int j = 0; j < p.groups; ++j) {
            const uint32_t o = __shfl_sync(kFull, score, j << p.llog);
            rank += (o > score || (o == score && j < grp)) ? 1 : 0;
        }
        if (rank >= p.topk_groups) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = 0u;
        }
    }

    int mine = 0;  // lane j: the j-th choice
    for (int j = 0; j < p.k; ++j) {
        uint32_t m = key[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) m = max(m, key[i]);
        const uint32_t top = __reduce_max_sync(kFull, m);
        const int from = __ffs(__ballot_sync(kFull, m == top)) - 1;
        int at = 0;
        bool open = lane == from;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            if (open && key[i] == top) {
                key[i] = 0u;
                at = i;
                open = false;
            }
        }
        const int e = __shfl_sync(kFull, first + at, from);
        if (lane == j) mine = e;
    }
    float s = 0.f;
    if (lane < p.k) {
        const float t = to_f32(x[mine]);
        s = p.sigmoid ? logistic(t) : expf(t - mx) / total;
    }
    float w = s * p.scale;
    if (p.renormalise) {
        const float sum = warp_sum_f32(s);
        w = sum > 0.f ? p.scale * s / sum : 0.f;
    }
    if (lane < p.k) {
        p.weights[row * p.k + lane] = w;
        p.experts[row * p.k + lane] = mine;
        if (p.counts) atomicAdd(p.counts + mine, 1);
    }
}

// ---------------------------------------------------------------- gradient ----------
// With D = sum of the chosen s, w^_j = s_j / D and g the gradient of the weights:
//   renormalised:  ds_j = scale * (g_j - sum_i g_i w^_i) / D,   else  ds_j = scale * g_j
//   sigmoid:       dx_j = ds_j s_j (1 - s_j)
//   softmax:       dx_e = s_e ([e chosen] ds_e - sum_j ds_j s_j); renormalised, the sum is
//                  zero and D cancels: dx_j = scale * w^_j (g_j - sum_i g_i w^_i), where w^ is
//                  the softmax of the chosen logits alone.
// The choice itself has no gradient, so neither has the bias.
// One warp per row: lane j < k holds choice j.  Every row of the output is written whole
// (zeros, or -s_e sum ds s for the softmax that is not renormalised), then, after a warp
// barrier, the chosen columns over it; both writes meet in L2.
struct RouteBackParams {
    const float* grad;
    const void* logits;
    const int32_t* experts;
    void* out;
    int64_t rows, row_stride, out_stride;
    int32_t E, k, sigmoid, renormalise;
    float scale;
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kRouteWarps * 32) ds_route_backward_kernel(const RouteBackParams p) {
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * kRouteWarps + (threadIdx.x >> 5);
    pdl_launch_dependents();
    pdl_wait();
    if (row >= p.rows) return;
    const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
    T* out = static_cast<T*>(p.out) + row * p.out_stride;
    int e = -1;
    float g = 0.f;
    if (lane < p.k) {
        e = p.experts[row * p.k + lane];
        if (e < 0 || e >= p.E) e = -1;  // not a column: it has no part
        g = p.grad[row * p.k + lane];
    }
    const bool on = e >= 0;
    if (!on) g = 0.f;
    const float t = on ? to_f32(x[e]) : -INFINITY;
    const bool whole = !p.sigmoid && !p.renormalise;  // every column has a gradient
    float mx = 0.f, total = 1.f;
    if (whole) {
        float m = -INFINITY;
        for (int c = lane; c < p.E; c += 32) m = fmaxf(m, to_f32(x[c]));
        mx = row_max(warp_max_f32(m));
        float s = 0.f;
        for (int c = lane; c < p.E; c += 32) s += expf(to_f32(x[c]) - mx);
        total = row_sum(warp_sum_f32(s));
    } else if (!p.sigmoid) {
        mx = row_max(warp_max_f32(t));
    }
    const float s = !on ? 0.f : p.sigmoid ? logistic(t) : expf(t - mx) / total;
    float d = p.scale * g, back = 0.f;
    if (p.renormalise) {
        const float sum = warp_sum_f32(s);
        const float inv = sum > 0.f ? 1.0f / sum : 0.f;
        const float mean = warp_sum_f32(g * s * inv);
        d = on ? p.scale * (g - mean) * inv : 0.f;
    }
    if (whole) back = warp_sum_f32(d * s);
    const float dx = p.sigmoid ? d * s * (1.0f - s) : s * (d - back);

    if (whole) {
        for (int c = lane; c < p.E; c += 32)
            out[c] = from_f32<T>(-back * (expf(to_f32(x[c]) - mx) / total));
    } else if (VEC) {
        constexpr int PER = 16 / sizeof(T);
        for (int c = lane; c < p.E / PER; c += 32) reinterpret_cast<uint4*>(out)[c] = make_uint4(0u, 0u, 0u, 0u);
    } else {
        for (int c = lane; c < p.E; c += 32) out[c] = from_f32<T>(0.f);
    }
    __syncwarp();
    if (on) out[e] = from_f32<T>(dx);
}

// ---------------------------------------------------------------- host --------------
template <typename T, bool VEC>
static ds_status launch_route(const RouteParams& p, int epl, cudaStream_t stream) {
    const dim3 grid(static_cast<unsigned>((p.rows + kRouteWarps - 1) / kRouteWarps));
    switch (epl) {
        case 1: return launch_pdl(ds_route_kernel<T, 1, VEC>, grid, kRouteWarps * 32, 0, 1, stream, p);
        case 2: return launch_pdl(ds_route_kernel<T, 2, VEC>, grid, kRouteWarps * 32, 0, 1, stream, p);
        case 4: return launch_pdl(ds_route_kernel<T, 4, VEC>, grid, kRouteWarps * 32, 0, 1, stream, p);
        case 8: return launch_pdl(ds_route_kernel<T, 8, VEC>, grid, kRouteWarps * 32, 0, 1, stream, p);
        case 16: return launch_pdl(ds_route_kernel<T, 16, VEC>, grid, kRouteWarps * 32, 0, 1, stream, p);
        default: return launch_pdl(ds_route_kernel<T, 32, VEC>, grid, kRouteWarps * 32, 0, 1, stream, p);
    }
}

}  // namespace dsk

using namespace dsk;

extern "C" {

ds_status ds_route(const void* logits, int32_t dtype, int64_t rows, int32_t E, int64_t row_stride, int32_t k,
                   int32_t scoring, const float* bias, int32_t groups, int32_t topk_groups, int32_t group_score,
                   int32_t renormalise, float scale, float* out_weights, int32_t* out_experts, int32_t* counts,
                   cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || rows < 0 || E < 1 || row_stride < E || k < 1) return DS_ERR_INVALID_ARG;
    if ((scoring != DS_SOFTMAX && scoring != DS_SIGMOID) || (group_score != DS_GROUP_MAX && group_score != DS_GROUP_TOP2))
        return DS_ERR_INVALID_ARG;
    if (groups < 1 || E % groups != 0 || topk_groups < 1 || topk_groups > groups) return DS_ERR_INVALID_ARG;
    if (k > static_cast<int64_t>(E / groups) * topk_groups || !isfinite(scale)) return DS_ERR_INVALID_ARG;
    if (E > kRouteMaxE || k > kRouteMaxK || groups > 32) return DS_ERR_UNSUPPORTED;
    if ((rows + kRouteWarps - 1) / kRouteWarps > 0x7FFFFFFFLL) return DS_ERR_UNSUPPORTED;
    if (rows == 0) return DS_OK;
    if (!logits || !out_weights || !out_experts) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(logits);
    if (bits % es || reinterpret_cast<uintptr_t>(bias) % 4 || reinterpret_cast<uintptr_t>(out_weights) % 4 ||
        reinterpret_cast<uintptr_t>(out_experts) % 4 || reinterpret_cast<uintptr_t>(counts) % 4)
        return DS_ERR_ALIGNMENT;
    RouteParams p = {};
    p.logits = logits;
    p.bias = bias;
    p.weights = out_weights;
    p.experts = out_experts;
    p.counts = counts;
    p.rows = rows;
    p.row_stride = row_stride;
    p.E = E;
    p.k = k;
    p.groups = groups;
    p.topk_groups = topk_groups;
    p.size = E / groups;
    while ((2 << p.llog) * groups <= 32) ++p.llog;
    p.n = (p.size + (1 << p.llog) - 1) >> p.llog;
    p.sigmoid = scoring == DS_SIGMOID;
    p.top2 = group_score == DS_GROUP_TOP2;
    p.renormalise = renormalise != 0;
    p.scale = scale;
    int epl = 1;
    while (epl < p.n) epl <<= 1;
    // 16-byte loads when every lane's run starts on 16 bytes; else element by element
    const bool vec = bits % 16 == 0 && row_stride * es % 16 == 0 && static_cast<int64_t>(p.n) * es % 16 == 0 &&
                     static_cast<int64_t>(p.size) * es % 16 == 0;
    if (dtype == DS_BF16)
        return vec ? launch_route<__nv_bfloat16, true>(p, epl, stream) : launch_route<__nv_bfloat16, false>(p, epl, stream);
    return vec ? launch_route<float, true>(p, epl, stream) : launch_route<float, false>(p, epl, stream);
}

ds_status ds_route_backward(const float* grad_weights, const void* logits, int32_t dtype, int64_t rows, int32_t E,
                            int64_t row_stride, int32_t k, const int32_t* experts, int32_t scoring,
                            int32_t renormalise, float scale, void* grad_logits, int64_t grad_stride,
                            cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || rows < 0 || E < 1 || row_stride < E || grad_stride < E || k < 1 || k > E)
        return DS_ERR_INVALID_ARG;
    if ((scoring != DS_SOFTMAX && scoring != DS_SIGMOID) || !isfinite(scale)) return DS_ERR_INVALID_ARG;
    if (E > kRouteMaxE || k > kRouteMaxK) return DS_ERR_UNSUPPORTED;
    if ((rows + kRouteWarps - 1) / kRouteWarps > 0x7FFFFFFFLL) return DS_ERR_UNSUPPORTED;
    if (rows == 0) return DS_OK;
    if (!grad_weights || !logits || !experts || !grad_logits) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    const uintptr_t gb = reinterpret_cast<uintptr_t>(grad_logits);
    if (reinterpret_cast<uintptr_t>(logits) % es || gb % es || reinterpret_cast<uintptr_t>(grad_weights) % 4 ||
        reinterpret_cast<uintptr_t>(experts) % 4)
        return DS_ERR_ALIGNMENT;
    const RouteBackParams p = {grad_weights, logits, experts, grad_logits, rows, row_stride, grad_stride,
                               E, k, scoring == DS_SIGMOID, renormalise != 0, scale};
    const bool vec = gb % 16 == 0 && grad_stride * es % 16 == 0 && static_cast<int64_t>(E) * es % 16 == 0;
    const dim3 grid(static_cast<unsigned>((rows + kRouteWarps - 1) / kRouteWarps));
    const int threads = kRouteWarps * 32;
    if (dtype == DS_BF16)
        return vec ? launch_pdl(ds_route_backward_kernel<__nv_bfloat16, true>, grid, threads, 0, 1, stream, p)
                   : launch_pdl(ds_route_backward_kernel<__nv_bfloat16, false>, grid, threads, 0, 1, stream, p);
    return vec ? launch_pdl(ds_route_backward_kernel<float, true>, grid, threads, 0, 1, stream, p)
               : launch_pdl(ds_route_backward_kernel<float, false>, grid, threads, 0, 1, stream, p);
}

}  // extern "C"
