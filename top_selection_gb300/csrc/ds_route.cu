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
// lowest lane holding a maximum holds the lowest expert.  Each lane sorts its order-preserving
// integer keys (lists of up to 8, by a network of minima and maxima); selection is then k rounds
// of: largest head of the warp (redux.sync), lowest lane that has it (ballot), and that lane moves
// its list up.  Lane j < k keeps the j-th choice's key and holder, and looks the expert up among
// the holder's unsorted keys at the end, all choices at once.  (Instructions for a row of 256
// experts: searching unsorted lanes in every round 1172, sorting pairs of key and place 996, keys
// alone with equal choices counted in every round 928, counted at the end 879.)
// It reads its expert's logit again (the row is in L1) and computes its weight.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kRouteWarps = 8;     // rows at a time per CTA
// The same where choices are counted, and such CTAs on an SM.  With 8 or 16 experts a lane, cut to 56
// registers, 36 warps find room in three CTAs (16384 rows of 256 in groups, with gradient: 23.8 us, two
// of 16 warps 25.3; 512 experts, which spill 32 to 44 bytes a thread then, 42.2 and 44.8); with fewer, two CTAs have their counts cleared and added
// sooner (8190 rows of 60 experts: 7.1 us, three of 12 warps 8.2).
template <int EPL>
constexpr int kCountWarps = EPL == 8 || EPL == 16 ? 12 : 16;
template <int EPL>
constexpr int kCountCtas = EPL < 8 ? 2 : EPL < 32 ? 3 : 1;
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

// exp(x) for sums of many terms, off by 2^-22 of each; a chosen expert's own term goes by expf.
__device__ __forceinline__ float exp_term(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
    return r;
}

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

// Sorts L numbers, the largest first (odd-even merge networks).
__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
    const uint32_t hi = max(a, b), lo = min(a, b);
    a = hi;
    b = lo;
}
template <int L>
__device__ __forceinline__ void sort_down(uint32_t (&x)[L]) {
    if constexpr (L == 2) {
        order(x[0], x[1]);
    } else if constexpr (L == 4) {
        order(x[0], x[1]), order(x[2], x[3]), order(x[0], x[2]), order(x[1], x[3]), order(x[1], x[2]);
    } else if constexpr (L == 8) {
        order(x[0], x[1]), order(x[2], x[3]), order(x[4], x[5]), order(x[6], x[7]);
        order(x[0], x[2]), order(x[1], x[3]), order(x[4], x[6]), order(x[5], x[7]);
        order(x[1], x[2]), order(x[5], x[6]);
        order(x[0], x[4]), order(x[1], x[5]), order(x[2], x[6]), order(x[3], x[7]);
        order(x[2], x[4]), order(x[3], x[5]);
        order(x[1], x[2]), order(x[3], x[4]), order(x[5], x[6]);
    }
}

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
__device__ __forceinline__ void route_row(const RouteParams& p, int64_t row, int lane, int* count_in) {
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
        for (int i = 0; i < EPL; ++i) s += i < count ? exp_term(v[i] - mx) : 0.f;
        total = row_sum(warp_sum_f32(s));
    }
    // choice values; places past the run get key 0, below every value's key
    uint32_t key[EPL];
    if (p.bias) {
        float b[EPL];
        load_run<float, EPL, VEC>(p.bias + (count > 0 ? first : 0), count, 0.f, b);
#pragma unroll
        for (int i = 0; i < EPL; ++i) v[i] = (p.sigmoid ? logistic(v[i]) : expf(v[i] - mx) / total) + b[i];
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
        score = grp < p.groups ? max(score, 1u) : 0u;  // lanes behind the last group have none
        bool keep = false;
        for (int j = 0; j < p.topk_groups; ++j) {  // the best group, the lowest of equal ones, in turn
            const uint32_t top = __reduce_max_sync(kFull, score);
            const int from = __ffs(__ballot_sync(kFull, score == top)) - 1;
            if (grp == from >> p.llog) {
                keep = true;
                score = 0u;
            }
        }
        if (!keep) {
#pragma unroll
            for (int i = 0; i < EPL; ++i) key[i] = 0u;
        }
    }

    // each lane's keys in sorted lists; then k rounds of the warp's largest head
    constexpr int L = EPL < 8 ? EPL : 8, NL = EPL / L;
    uint32_t list[NL][L];
#pragma unroll
    for (int n = 0; n < NL; ++n) {
#pragma unroll
        for (int i = 0; i < L; ++i) list[n][i] = key[n * L + i];
        sort_down<L>(list[n]);
    }
    // lane j: the j-th choice's key and the lane that holds it
    uint32_t won = 0u;
    int holder = lane;
    for (int j = 0; j < p.k; ++j) {
        uint32_t head = list[0][0];
#pragma unroll
        for (int n = 1; n < NL; ++n) head = max(head, list[n][0]);
        const uint32_t top = __reduce_max_sync(kFull, head);
        const int from = __ffs(__ballot_sync(kFull, head == top)) - 1;
        if (lane == j) {
            won = top;
            holder = from;
        }
        bool open = lane == from;
#pragma unroll
        for (int n = 0; n < NL; ++n) {
            const bool here = open && (n == NL - 1 || list[n][0] == top);
#pragma unroll
            for (int i = 0; i + 1 < L; ++i) list[n][i] = here ? list[n][i + 1] : list[n][i];
            list[n][L - 1] = here ? 0u : list[n][L - 1];
            open = open && !here;
        }
    }
    // the expert behind each choice: the holder's first place with that key, or one further for each
    // choice right before it with the same key and holder (a holder's equal keys come in turn)
    const uint32_t won_up = __shfl_up_sync(kFull, won, 1);
    const int holder_up = __shfl_up_sync(kFull, holder, 1);
    const uint32_t again = __ballot_sync(kFull, lane > 0 && won == won_up && holder == holder_up);
    int before = lane - (31 - __clz(~again & ((2u << lane) - 1u)));
    int mine = __shfl_sync(kFull, first, holder);
    {
        int at = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const bool hit = __shfl_sync(kFull, key[i], holder) == won;
            if (hit && before == 0) at = i;
            before -= hit ? 1 : 0;
        }
        mine += at;
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
        if (count_in) atomicAdd(count_in + mine, 1);
    }
}

// Choices are counted in shared memory and added to the caller's counts once per CTA (rows going
// straight to the counts meet in a few lines of L2: 131072 choices of 256 experts took 8 us).
template <typename T, int EPL, bool VEC, bool COUNT>
__global__ void __launch_bounds__((COUNT ? kCountWarps<EPL> : kRouteWarps) * 32, COUNT && kCountCtas<EPL> == 3 ? 3 : 0)
ds_route_kernel(const RouteParams p) {
    constexpr int WARPS = COUNT ? kCountWarps<EPL> : kRouteWarps;
    __shared__ int sh_count[COUNT ? kRouteMaxE : 1];
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    if (COUNT) {
        for (int e = threadIdx.x; e < p.E; e += WARPS * 32) sh_count[e] = 0;
        __syncthreads();
    }
    pdl_wait();
    for (int64_t row = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5); row < p.rows;
         row += static_cast<int64_t>(gridDim.x) * WARPS)
        route_row<T, EPL, VEC>(p, row, lane, COUNT ? sh_count : nullptr);
    if (COUNT) {
        __syncthreads();
        for (int e = threadIdx.x; e < p.E; e += WARPS * 32)
            if (sh_count[e]) atomicAdd(p.counts + e, sh_count[e]);
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
// LPR lanes per row (8 where k <= 8, so that a warp takes four rows): lane j < k holds choice j.
// Every row of the output is written whole, first zeros, or for the softmax that is not
// renormalised -s_e sum ds s, then, after a warp barrier, the chosen columns over them; both writes
// meet in L2.
struct RouteBackParams {
    const float* grad;
    const void* logits;
    const int32_t* experts;
    void* out;
    int64_t rows, row_stride, out_stride;
    int32_t E, k, sigmoid, renormalise;
    float scale;
};

template <int LPR>
__device__ __forceinline__ float part_sum(float v) {
#pragma unroll
    for (int d = LPR / 2; d >= 1; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
    return v;
}
template <int LPR>
__device__ __forceinline__ float part_max(float v) {
#pragma unroll
    for (int d = LPR / 2; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, d));
    return v;
}

// WHOLE: every column has a gradient (softmax, not renormalised); a lane holds up to NPL of them.
// VEC: otherwise, the zeros may be written 16 bytes at a time.
template <typename T, int LPR, int NPL, bool WHOLE, bool VEC>
__global__ void __launch_bounds__(kRouteWarps * 32) ds_route_backward_kernel(const RouteBackParams p) {
    const int lane = threadIdx.x & 31, sub = lane % LPR;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * (kRouteWarps * 32 / LPR) + threadIdx.x / LPR;
    pdl_launch_dependents();
    pdl_wait();
    const bool live = at < p.rows;  // the warp stays whole for its shuffles
    const int64_t row = live ? at : p.rows - 1;
    const T* x = static_cast<const T*>(p.logits) + row * p.row_stride;
    T* out = static_cast<T*>(p.out) + row * p.out_stride;
    int e = -1;
    float g = 0.f;
    if (sub < p.k) {
        e = p.experts[row * p.k + sub];
        if (e < 0 || e >= p.E) e = -1;  // not a column: it has no part
        g = p.grad[row * p.k + sub];
    }
    float v[NPL];
    float mx = 0.f, total = 1.f;
    if (WHOLE) {
        float m = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int c = sub + i * LPR;
            v[i] = c < p.E ? to_f32(x[c]) : -INFINITY;
            m = fmaxf(m, v[i]);
        }
        mx = row_max(part_max<LPR>(m));
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            v[i] = exp_term(v[i] - mx);
            s += v[i];
        }
        total = row_sum(part_sum<LPR>(s));
    }
    const bool on = e >= 0;
    if (!on) g = 0.f;
    const float t = on ? to_f32(x[e]) : -INFINITY;
    if (!WHOLE && !p.sigmoid) mx = row_max(part_max<LPR>(t));
    const float s = !on ? 0.f : p.sigmoid ? logistic(t) : expf(t - mx) / total;
    // d w is s ds without 1 / D by itself: logistic scores may be so small that it is infinite
    float d = p.scale * g, back = 0.f, w = s;
    if (p.renormalise) {
        const float sum = part_sum<LPR>(s);
        w = sum > 0.f ? s / sum : 0.f;
        d = p.scale * (g - part_sum<LPR>(g * w));
    }
    if (WHOLE) back = part_sum<LPR>(d * s);
    const float dx = p.sigmoid ? d * w * (1.0f - s) : w * (d - back);
    if (live) {
        if (WHOLE) {
            const float f = -back / total;
#pragma unroll
            for (int i = 0; i < NPL; ++i)
                if (sub + i * LPR < p.E) out[sub + i * LPR] = from_f32<T>(f * v[i]);
        } else if (VEC) {
            constexpr int PER = 16 / sizeof(T);
            for (int c = sub; c < p.E / PER; c += LPR) reinterpret_cast<uint4*>(out)[c] = make_uint4(0u, 0u, 0u, 0u);
        } else {
            for (int c = sub; c < p.E; c += LPR) out[c] = from_f32<T>(0.f);
        }
    }
    __syncwarp();
    if (live && on) out[e] = from_f32<T>(dx);
}

// ---------------------------------------------------------------- host --------------
template <typename T, int EPL, bool VEC>
static ds_status launch_route_as(const RouteParams& p, int sms, cudaStream_t stream) {
    if (!p.counts) {
        const int64_t ctas = (p.rows + kRouteWarps - 1) / kRouteWarps;
        return launch_pdl(ds_route_kernel<T, EPL, VEC, false>, dim3(static_cast<unsigned>(ctas)), kRouteWarps * 32, 0, 1,
                          stream, p);
    }
    // as many CTAs as fit at once, each for many rows: the counts are added once per CTA
    constexpr int WARPS = kCountWarps<EPL>;
    int64_t ctas = (p.rows + WARPS - 1) / WARPS;
    const int64_t most = static_cast<int64_t>(sms) * kCountCtas<EPL>;
    if (ctas > most) ctas = most;
    return launch_pdl(ds_route_kernel<T, EPL, VEC, true>, dim3(static_cast<unsigned>(ctas)), WARPS * 32, 0, 1, stream, p);
}

// 16-byte loads exist where a lane's run holds 16 bytes
template <typename T>
static ds_status launch_route(const RouteParams& p, int epl, bool vec, int sms, cudaStream_t stream) {
    constexpr bool WIDE = sizeof(T) == 4;
    switch (epl) {
        case 1: return launch_route_as<T, 1, false>(p, sms, stream);
        case 2: return launch_route_as<T, 2, false>(p, sms, stream);
        case 4: return vec && WIDE ? launch_route_as<T, 4, WIDE>(p, sms, stream) : launch_route_as<T, 4, false>(p, sms, stream);
        case 8: return vec ? launch_route_as<T, 8, true>(p, sms, stream) : launch_route_as<T, 8, false>(p, sms, stream);
        case 16: return vec ? launch_route_as<T, 16, true>(p, sms, stream) : launch_route_as<T, 16, false>(p, sms, stream);
        default: return vec ? launch_route_as<T, 32, true>(p, sms, stream) : launch_route_as<T, 32, false>(p, sms, stream);
    }
}

template <typename T>
static ds_status launch_route_backward(const RouteBackParams& p, bool vec, cudaStream_t stream) {
    const bool whole = !p.sigmoid && !p.renormalise, narrow = p.k <= 8 && (!whole || p.E <= 64);
    const int rows = kRouteWarps * 32 / (narrow ? 8 : 32);
    const dim3 grid(static_cast<unsigned>((p.rows + rows - 1) / rows));
    const auto go = [&](auto kern) { return launch_pdl(kern, grid, kRouteWarps * 32, 0, 1, stream, p); };
    if (whole) {
        if (narrow) return go(ds_route_backward_kernel<T, 8, 8, true, false>);
        return p.E <= 256 ? go(ds_route_backward_kernel<T, 32, 8, true, false>) : go(ds_route_backward_kernel<T, 32, 16, true, false>);
    }
    if (narrow) return vec ? go(ds_route_backward_kernel<T, 8, 1, false, true>) : go(ds_route_backward_kernel<T, 8, 1, false, false>);
    return vec ? go(ds_route_backward_kernel<T, 32, 1, false, true>) : go(ds_route_backward_kernel<T, 32, 1, false, false>);
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
    if (rows > 0x7FFFFFFFLL * kRouteWarps) return DS_ERR_UNSUPPORTED;
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
    // 16-byte loads when every lane's run (and its bias) starts on 16 bytes; else element by element
    const bool vec = bits % 16 == 0 && row_stride * es % 16 == 0 && static_cast<int64_t>(p.n) * es % 16 == 0 &&
                     static_cast<int64_t>(p.size) * es % 16 == 0 && aligned16(bias);
    int dev = 0;
    DevInfo info;
    if (cudaGetDevice(&dev) != cudaSuccess || !dev_info(dev, info)) return DS_ERR_CUDA;
    return dtype == DS_BF16 ? launch_route<__nv_bfloat16>(p, epl, vec, info.sms, stream)
                            : launch_route<float>(p, epl, vec, info.sms, stream);
}

ds_status ds_route_backward(const float* grad_weights, const void* logits, int32_t dtype, int64_t rows, int32_t E,
                            int64_t row_stride, int32_t k, const int32_t* experts, int32_t scoring,
                            int32_t renormalise, float scale, void* grad_logits, int64_t grad_stride,
                            cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || rows < 0 || E < 1 || row_stride < E || grad_stride < E || k < 1 || k > E)
        return DS_ERR_INVALID_ARG;
    if ((scoring != DS_SOFTMAX && scoring != DS_SIGMOID) || !isfinite(scale)) return DS_ERR_INVALID_ARG;
    if (E > kRouteMaxE || k > kRouteMaxK) return DS_ERR_UNSUPPORTED;
    if (rows > 0x7FFFFFFFLL * kRouteWarps) return DS_ERR_UNSUPPORTED;
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
    return dtype == DS_BF16 ? launch_route_backward<__nv_bfloat16>(p, vec, stream) : launch_route_backward<float>(p, vec, stream);
}

}  // extern "C"
