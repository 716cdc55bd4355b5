// ds_experts.cu -- the exchange behind the experts' gate: choices sorted by expert
// (ds_expert_sort), tokens brought into that order (ds_expert_gather; in 8 bits by
// ds_quantise.cu), the experts' outputs back with the gate's weights (ds_expert_combine), and
// the gradient of that sum (ds_expert_combine_backward).
//
// Slot s = t k + i is token t's i-th choice.  place[s] is its rank among all slots that have an
// expert, by expert, then by slot; offsets[e] is the first place of expert e.  Then
//   gather:   rows[place[t, i]] = x[t]
//   combine:  out[t] = sum_i w[t, i] y[place[t, i]]
//   backward: dy[place[t, i]] = w[t, i] g[t],  dw[t, i] = g[t] . y[place[t, i]]
// and gather's gradient is combine without weights.  Every kernel works from the token's side, which
// reads (or writes) a token's row once, not once for each of its choices.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_rows.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kSortWarps = 32;
constexpr int kSortCluster = 16;
constexpr int kSortMaxE = 512;
constexpr int kMaxChoices = 32;    // one lane per choice
constexpr uint32_t kEvery = 0xFFFFFFFFu;

// ---------------------------------------------------------------- sort --------------
// A counting sort in one launch: one cluster, each CTA a run of the slots, each warp a run of the
// CTA's.  Warps count their experts in shared memory, the counts are summed over a CTA's warps and
// over the cluster (distributed shared memory) into each warp's first place for each expert, and
// each warp goes over its slots again in order, 32 at a time: equal experts among them (match) are
// ranked by lane.  Ranks depend on no order of atomics: places are the stable sort's.
struct SortParams {
    const int32_t* experts;
    int32_t* places;
    int32_t* offsets;
    int64_t slots;
    int64_t per_cta, per_warp;
    int32_t E;
    int32_t warps;   // warps of a CTA that have slots
};

__global__ void __launch_bounds__(kSortWarps * 32) ds_expert_sort_kernel(const SortParams p) {
    extern __shared__ int32_t sh_count[];  // [warps][E]
    __shared__ int32_t sh_total[kSortMaxE], sh_first[kSortMaxE], sh_scan[kSortWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = blockIdx.x, ctas = gridDim.x;
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < p.warps * p.E; i += blockDim.x) sh_count[i] = 0;
    __syncthreads();
    pdl_wait();
    const int64_t cta_end = min(p.slots, (rank + 1) * p.per_cta);
    const int64_t begin = rank * p.per_cta + warp * p.per_warp;
    const int64_t end = min(cta_end, begin + p.per_warp);
    int32_t* mine = sh_count + warp * p.E;
    if (warp < p.warps)
        for (int64_t s = begin + lane; s < end; s += 32) {
            const int e = p.experts[s];
            if (e >= 0 && e < p.E) atomicAdd(mine + e, 1);
        }
    __syncthreads();
    // counts -> places before the warp's own within the CTA's
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
        int sum = 0;
#pragma unroll 8
        for (int w = 0; w < p.warps; ++w) {
            const int c = sh_count[w * p.E + e];
            sh_count[w * p.E + e] = sum;
            sum += c;
        }
        sh_total[e] = sum;
    }
    if (ctas > 1) cluster_sync_all();
    else __syncthreads();
    int before = 0, total = 0;  // thread e: the expert's slots in earlier CTAs, and in all
    const int e = threadIdx.x;
    if (e < p.E) {
        if (ctas > 1) {
            for (uint32_t r = 0; r < ctas; ++r) {
                const int c = static_cast<int>(ld_cluster_u32(map_rank(&sh_total[e], r)));
                before += r < rank ? c : 0;
                total += c;
            }
        } else {
            total = sh_total[e];
        }
    }
    const int upto = static_cast<int>(warp_incl_scan(static_cast<uint32_t>(total), lane));
    if (lane == 31) sh_scan[warp] = upto;
    __syncthreads();
    if (e < p.E) {
        int first = upto - total;
        for (int w = 0; w < warp; ++w) first += sh_scan[w];
        sh_first[e] = first + before;
        if (rank == 0) {
            p.offsets[e] = first;
            if (e == p.E - 1) p.offsets[p.E] = first + total;
        }
    }
    if (ctas > 1) cluster_sync_all();  // also: no CTA leaves while its totals are read
    else __syncthreads();
    if (warp >= p.warps) return;
    for (int64_t s0 = begin; s0 < end; s0 += 32) {
        const int64_t s = s0 + lane;
        int x = s < end ? p.experts[s] : -1;
        if (x < 0 || x >= p.E) x = -1;
        const uint32_t same = __match_any_sync(kEvery, x);
        const int behind = __popc(same & lanemask_lt());
        int at = 0;
        if (x >= 0) at = mine[x];
        __syncwarp();
        if (x >= 0 && behind == 0) mine[x] = at + __popc(same);
        __syncwarp();
        if (s < end) p.places[s] = x >= 0 ? sh_first[x] + at + behind : -1;
    }
}

// ---------------------------------------------------------------- rows --------------
// WPR warps to a token's row, 8 warps to a CTA; a thread takes 16 bytes at a time (VEC), or one
// number where rows do not start on 16 bytes.  Lane i of each warp keeps the token's i-th place.
constexpr int kRowWarps = 8;

// The place of the lane's choice, -1 for none.
__device__ __forceinline__ int64_t place_of(const int32_t* places, int64_t token, int k, int lane, int64_t rows) {
    if (lane >= k) return -1;
    const int64_t at = places[token * k + lane];
    return at < rows ? at : -1;
}

struct GatherParams {
    const void* x;
    const int32_t* places;
    const int32_t* offsets;
    void* out;
    int64_t tokens, stride;
    int32_t D, k, E;
};

template <typename T, int WPR, bool VEC>
__global__ void __launch_bounds__(kRowWarps * 32) ds_expert_gather_kernel(const GatherParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t token = static_cast<int64_t>(blockIdx.x) * (kRowWarps / WPR) + warp / WPR;
    if (token >= p.tokens) return;
    const int64_t rows = p.tokens * p.k;
    const int64_t place = place_of(p.places, token, p.k, lane, rows);
    const int64_t filled = p.offsets[p.E];
    using Word = typename std::conditional<VEC, uint4, T>::type;
    const int n = VEC ? p.D / kPer<T> : p.D;
    const Word* src = reinterpret_cast<const Word*>(static_cast<const T*>(p.x) + token * p.stride);
    T* out = static_cast<T*>(p.out);
    constexpr int STEP = WPR * 32, U = 4;
    for (int c = (warp % WPR) * 32 + lane; __any_sync(kEvery, c < n); c += STEP * U) {
        Word v[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c + u * STEP < n) v[u] = src[c + u * STEP];
        for (int i = 0; i < p.k; ++i) {
            const int64_t at = __shfl_sync(kEvery, place, i);
            if (at < 0) continue;
            Word* dst = reinterpret_cast<Word*>(out + at * p.D);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c + u * STEP < n) dst[c + u * STEP] = v[u];
        }
    }
    // rows behind the last expert's: zeros, as many as slots are without an expert
    for (int64_t r = max(filled, token * p.k); r < (token + 1) * p.k; ++r) {
        Word* dst = reinterpret_cast<Word*>(out + r * p.D);
        for (int c = (warp % WPR) * 32 + lane; c < n; c += STEP) {
            if constexpr (VEC) dst[c] = make_uint4(0u, 0u, 0u, 0u);
            else row_put(dst + c, 0.f);
        }
    }
}

struct CombineParams {
    const void* y;
    const int32_t* places;
    const float* weights;
    void* out;
    int64_t tokens, rows, stride;
    int32_t D, k;
};

template <typename T, int WPR, bool VEC>
__global__ void __launch_bounds__(kRowWarps * 32) ds_expert_combine_kernel(const CombineParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t token = static_cast<int64_t>(blockIdx.x) * (kRowWarps / WPR) + warp / WPR;
    if (token >= p.tokens) return;
    const int64_t place = place_of(p.places, token, p.k, lane, p.rows);
    float weight = 1.f;
    if (p.weights && lane < p.k) weight = p.weights[token * p.k + lane];
    const T* y = static_cast<const T*>(p.y);
    T* out = static_cast<T*>(p.out) + token * p.D;
    constexpr int STEP = WPR * 32, U = 8, PER = VEC ? kPer<T> : 1;  // U rows at a time
    const int n = p.D / PER;
    for (int c = (warp % WPR) * 32 + lane; __any_sync(kEvery, c < n); c += STEP) {
        const bool in = c < n;
        float sum[PER] = {};
        for (int i0 = 0; i0 < p.k; i0 += U) {
            if constexpr (VEC) {
                uint4 v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t at = __shfl_sync(kEvery, place, (i0 + u) & 31);
                    v[u] = make_uint4(0u, 0u, 0u, 0u);
                    if (in && i0 + u < p.k && at >= 0) v[u] = reinterpret_cast<const uint4*>(y + at * p.stride)[c];
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float w = __shfl_sync(kEvery, weight, (i0 + u) & 31);
                    const int64_t at = __shfl_sync(kEvery, place, (i0 + u) & 31);
                    if (i0 + u < p.k && at >= 0) {
                        float f[PER];
                        unpack16(v[u], f);
#pragma unroll
                        for (int j = 0; j < PER; ++j) sum[j] = fmaf(w, f[j], sum[j]);
                    }
                }
            } else {
                float v[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int64_t at = __shfl_sync(kEvery, place, (i0 + u) & 31);
                    v[u] = 0.f;
                    if (in && i0 + u < p.k && at >= 0) v[u] = row_f32(y[at * p.stride + c]);
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float w = __shfl_sync(kEvery, weight, (i0 + u) & 31);
                    const int64_t at = __shfl_sync(kEvery, place, (i0 + u) & 31);
                    if (i0 + u < p.k && at >= 0) sum[0] = fmaf(w, v[u], sum[0]);
                }
            }
        }
        if (in) {
            if constexpr (VEC) reinterpret_cast<uint4*>(out)[c] = pack16(sum);
            else row_put(out + c, sum[0]);
        }
    }
}

struct CombineBackParams {
    const void* grad;
    const void* y;
    const int32_t* places;
    const int32_t* offsets;
    const float* weights;
    void* grad_y;
    float* grad_weights;
    int64_t tokens, grad_stride, stride;
    int32_t D, k, E;
};

// KC: the most choices; a lane sums its part of each choice's product over the whole row, and the
// lanes' (and warps') parts are added at the end, in a fixed order.
template <typename T, int WPR, int KC, bool VEC>
__global__ void __launch_bounds__(kRowWarps * 32) ds_expert_combine_backward_kernel(const CombineBackParams p) {
    __shared__ float sh_part[kRowWarps][KC];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t token = static_cast<int64_t>(blockIdx.x) * (kRowWarps / WPR) + warp / WPR;
    if (WPR == 1 && token >= p.tokens) return;  // (a whole CTA has one token otherwise)
    const int64_t rows = p.tokens * p.k;
    const int64_t place = place_of(p.places, token, p.k, lane, rows);
    const int64_t filled = p.offsets[p.E];
    const float weight = lane < p.k ? p.weights[token * p.k + lane] : 0.f;
    const T* g = static_cast<const T*>(p.grad) + token * p.grad_stride;
    const T* y = static_cast<const T*>(p.y);
    T* gy = static_cast<T*>(p.grad_y);
    constexpr int STEP = WPR * 32, PER = VEC ? kPer<T> : 1;
    const int n = p.D / PER;
    float dot[KC] = {};
    for (int c = (warp % WPR) * 32 + lane; __any_sync(kEvery, c < n); c += STEP) {
        const bool in = c < n;
        float gv[PER];
        if constexpr (VEC) unpack16(in ? reinterpret_cast<const uint4*>(g)[c] : make_uint4(0u, 0u, 0u, 0u), gv);
        else gv[0] = in ? row_f32(g[c]) : 0.f;
        constexpr int U = KC < 8 ? KC : 8;
#pragma unroll
        for (int i0 = 0; i0 < KC; i0 += U) {
            if (i0 >= p.k) break;
            uint4 v[U];
            float f[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = __shfl_sync(kEvery, place, i0 + u);
                v[u] = make_uint4(0u, 0u, 0u, 0u), f[u] = 0.f;
                if (in && at >= 0) {
                    if constexpr (VEC) v[u] = reinterpret_cast<const uint4*>(y + at * p.stride)[c];
                    else f[u] = row_f32(y[at * p.stride + c]);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t at = __shfl_sync(kEvery, place, i0 + u);
                const float w = __shfl_sync(kEvery, weight, i0 + u);
                if (!in || at < 0) continue;
                if constexpr (VEC) {
                    float yv[PER], out[PER];
                    unpack16(v[u], yv);
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        dot[i0 + u] = fmaf(gv[j], yv[j], dot[i0 + u]);
                        out[j] = w * gv[j];
                    }
                    reinterpret_cast<uint4*>(gy + at * p.D)[c] = pack16(out);
                } else {
                    dot[i0 + u] = fmaf(gv[0], f[u], dot[i0 + u]);
                    row_put(gy + at * p.D + c, w * gv[0]);
                }
            }
        }
    }
    for (int64_t r = max(filled, token * p.k); r < (token + 1) * p.k; ++r)
        for (int c = (warp % WPR) * 32 + lane; c < n; c += STEP) {
            if constexpr (VEC) reinterpret_cast<uint4*>(gy + r * p.D)[c] = make_uint4(0u, 0u, 0u, 0u);
            else row_put(gy + r * p.D + c, 0.f);
        }
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < KC; ++i) {
        const float s = lanes_sum<32>(dot[i]);
        if (lane == i) mine = s;
    }
    if (WPR > 1) {
        if (lane < KC) sh_part[warp][lane] = mine;
        __syncthreads();
        if (warp > 0) return;
        mine = 0.f;
        if (lane < KC)
            for (int w = 0; w < WPR; ++w) mine += sh_part[w][lane];
    }
    if (lane < p.k) p.grad_weights[token * p.k + lane] = place >= 0 ? mine : 0.f;
}

// ---------------------------------------------------------------- host --------------
static bool aligned_rows(const void* p, int64_t stride, int64_t D, int es) {
    return aligned16(p) && stride * es % 16 == 0 && D * es % 16 == 0;
}

// One warp to a row where tokens are many (fewer sums over lanes), eight where they would leave most of
// the SMs' warps without a row.
static bool whole_cta(int64_t tokens, int sms) { return tokens < static_cast<int64_t>(sms) * 32; }

template <typename P, typename K1, typename K8>
static ds_status launch_rows(const P& p, int64_t tokens, int sms, cudaStream_t stream, K1 one, K8 eight) {
    const bool whole = whole_cta(tokens, sms);
    const int64_t ctas = whole ? tokens : (tokens + kRowWarps - 1) / kRowWarps;
    const dim3 grid(static_cast<unsigned>(ctas));
    return whole ? launch_pdl(eight, grid, kRowWarps * 32, 0, 1, stream, p)
                 : launch_pdl(one, grid, kRowWarps * 32, 0, 1, stream, p);
}

template <typename T>
static ds_status launch_gather(const GatherParams& p, bool vec, int sms, cudaStream_t s) {
    return vec ? launch_rows(p, p.tokens, sms, s, ds_expert_gather_kernel<T, 1, true>, ds_expert_gather_kernel<T, 8, true>)
               : launch_rows(p, p.tokens, sms, s, ds_expert_gather_kernel<T, 1, false>, ds_expert_gather_kernel<T, 8, false>);
}

template <typename T>
static ds_status launch_combine(const CombineParams& p, bool vec, int sms, cudaStream_t s) {
    return vec ? launch_rows(p, p.tokens, sms, s, ds_expert_combine_kernel<T, 1, true>, ds_expert_combine_kernel<T, 8, true>)
               : launch_rows(p, p.tokens, sms, s, ds_expert_combine_kernel<T, 1, false>, ds_expert_combine_kernel<T, 8, false>);
}

template <typename T, int KC>
static ds_status launch_combine_backward_as(const CombineBackParams& p, bool vec, int sms, cudaStream_t s) {
    return vec ? launch_rows(p, p.tokens, sms, s, ds_expert_combine_backward_kernel<T, 1, KC, true>,
                             ds_expert_combine_backward_kernel<T, 8, KC, true>)
               : launch_rows(p, p.tokens, sms, s, ds_expert_combine_backward_kernel<T, 1, KC, false>,
                             ds_expert_combine_backward_kernel<T, 8, KC, false>);
}

template <typename T>
static ds_status launch_combine_backward(const CombineBackParams& p, bool vec, int sms, cudaStream_t s) {
    if (p.k <= 2) return launch_combine_backward_as<T, 2>(p, vec, sms, s);
    if (p.k <= 4) return launch_combine_backward_as<T, 4>(p, vec, sms, s);
    if (p.k <= 8) return launch_combine_backward_as<T, 8>(p, vec, sms, s);
    return launch_combine_backward_as<T, 32>(p, vec, sms, s);
}

static ds_status device_sms(int& sms) {
    int dev = 0;
    DevInfo info;
    if (cudaGetDevice(&dev) != cudaSuccess || !dev_info(dev, info)) return DS_ERR_CUDA;
    sms = info.sms;
    return DS_OK;
}

static ds_status check_exchange(int64_t tokens, int32_t k, int32_t D) {
    if (tokens < 0 || k < 1 || D < 1) return DS_ERR_INVALID_ARG;
    if (k > kMaxChoices || tokens > 0x7FFFFFFFLL / k) return DS_ERR_UNSUPPORTED;
    return DS_OK;
}

static bool off(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

}  // namespace dsk

using namespace dsk;

extern "C" {

ds_status ds_expert_sort(const int32_t* experts, int64_t tokens, int32_t k, int32_t E, int32_t* places,
                         int32_t* offsets, cudaStream_t stream) {
    if (E < 1) return DS_ERR_INVALID_ARG;
    if (const ds_status st = check_exchange(tokens, k, 1)) return st;
    if (E > kSortMaxE) return DS_ERR_UNSUPPORTED;
    if (!offsets || (tokens > 0 && (!experts || !places))) return DS_ERR_INVALID_ARG;
    if (off(experts, 4) || off(places, 4) || off(offsets, 4)) return DS_ERR_ALIGNMENT;
    SortParams p = {};
    p.experts = experts;
    p.places = places;
    p.offsets = offsets;
    p.slots = tokens * k;
    p.E = E;
    // a CTA for each 2048 slots (two steps of 32 a warp), up to 16
    int ctas = 1;
    while (ctas < kSortCluster && p.slots > static_cast<int64_t>(ctas) * 2048) ctas *= 2;
    p.per_cta = (p.slots + ctas - 1) / ctas;
    p.per_warp = ((p.per_cta + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    p.warps = p.per_warp > 0 ? static_cast<int32_t>((p.per_cta + p.per_warp - 1) / p.per_warp) : 0;
    const size_t smem = static_cast<size_t>(p.warps) * E * sizeof(int32_t);
    if (cudaFuncSetAttribute(ds_expert_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSortWarps * kSortMaxE * static_cast<int>(sizeof(int32_t))) != cudaSuccess ||
        cudaFuncSetAttribute(ds_expert_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return DS_ERR_CUDA;
    return launch_pdl(ds_expert_sort_kernel, dim3(ctas), kSortWarps * 32, smem, ctas, stream, p);
}

ds_status ds_expert_gather(const void* x, int32_t dtype, int64_t tokens, int32_t D, int64_t row_stride,
                           const int32_t* places, int32_t k, const int32_t* offsets, int32_t E, void* out,
                           cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || row_stride < D || E < 1) return DS_ERR_INVALID_ARG;
    if (const ds_status st = check_exchange(tokens, k, D)) return st;
    if (E > kSortMaxE) return DS_ERR_UNSUPPORTED;
    if (tokens == 0) return DS_OK;
    if (!x || !places || !offsets || !out) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    if (off(x, es) || off(out, es) || off(places, 4) || off(offsets, 4)) return DS_ERR_ALIGNMENT;
    const GatherParams p = {x, places, offsets, out, tokens, row_stride, D, k, E};
    const bool vec = aligned_rows(x, row_stride, D, es) && aligned16(out);
    int sms = 0;
    if (const ds_status st = device_sms(sms)) return st;
    return dtype == DS_BF16 ? launch_gather<__nv_bfloat16>(p, vec, sms, stream) : launch_gather<float>(p, vec, sms, stream);
}

ds_status ds_expert_combine(const void* y, int32_t dtype, int64_t rows, int32_t D, int64_t row_stride,
                            const int32_t* places, int64_t tokens, int32_t k, const float* weights, void* out,
                            cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || rows < 0 || row_stride < D) return DS_ERR_INVALID_ARG;
    if (const ds_status st = check_exchange(tokens, k, D)) return st;
    if (tokens == 0) return DS_OK;
    if ((!y && rows > 0) || !places || !out) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    if (off(y, es) || off(out, es) || off(places, 4) || off(weights, 4)) return DS_ERR_ALIGNMENT;
    const CombineParams p = {y, places, weights, out, tokens, rows, row_stride, D, k};
    const bool vec = aligned_rows(y, row_stride, D, es) && aligned16(out);
    int sms = 0;
    if (const ds_status st = device_sms(sms)) return st;
    return dtype == DS_BF16 ? launch_combine<__nv_bfloat16>(p, vec, sms, stream) : launch_combine<float>(p, vec, sms, stream);
}

ds_status ds_expert_combine_backward(const void* grad, int64_t grad_stride, const void* y, int32_t dtype, int32_t D,
                                     int64_t row_stride, const int32_t* places, int64_t tokens, int32_t k,
                                     const int32_t* offsets, int32_t E, const float* weights, void* grad_y,
                                     float* grad_weights, cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || row_stride < D || grad_stride < D || E < 1) return DS_ERR_INVALID_ARG;
    if (const ds_status st = check_exchange(tokens, k, D)) return st;
    if (E > kSortMaxE) return DS_ERR_UNSUPPORTED;
    if (tokens == 0) return DS_OK;
    if (!grad || !y || !places || !offsets || !weights || !grad_y || !grad_weights) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    if (off(grad, es) || off(y, es) || off(grad_y, es) || off(places, 4) || off(offsets, 4) || off(weights, 4) ||
        off(grad_weights, 4))
        return DS_ERR_ALIGNMENT;
    const CombineBackParams p = {grad, y, places, offsets, weights, grad_y, grad_weights, tokens, grad_stride, row_stride,
                                 D, k, E};
    const bool vec = aligned_rows(grad, grad_stride, D, es) && aligned_rows(y, row_stride, D, es) && aligned16(grad_y);
    int sms = 0;
    if (const ds_status st = device_sms(sms)) return st;
    return dtype == DS_BF16 ? launch_combine_backward<__nv_bfloat16>(p, vec, sms, stream)
                            : launch_combine_backward<float>(p, vec, sms, stream);
}

}  // extern "C"
