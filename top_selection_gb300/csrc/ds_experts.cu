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
//
// Bound by memory where rows are long and many: 16384 tokens of 2048 bf16 numbers with 8 choices are gathered
// in 97 us (6.2 TB/s), combined in 90 (6.7) and go backward in 172 (6.6).  8190 x 4 rows of 1001 bf16 numbers,
// which start on 2 bytes only, run at 4.5, 4.0 and 4.3 TB/s: eight times as many words.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_rows.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kSortWarps = 32;
constexpr int kSortCluster = 16;
constexpr int kSortMaxE = 512;
constexpr int kMaxChoices = 32;    // one lane per choice
constexpr int kMaxColumns = 1 << 30;  // counted in 32 bits, a CTA's stretch of a row past the last one
constexpr uint32_t kEvery = 0xFFFFFFFFu;

// ---------------------------------------------------------------- sort --------------
// A counting sort in one launch: one cluster, each CTA a run of the slots, each warp a run of the
// CTA's.  Warps count their experts in shared memory, the counts are summed over a CTA's warps and
// over the cluster (distributed shared memory) into each warp's first place for each expert, and
// each warp goes over its slots again in order, 32 at a time: equal experts among them (match) are
// ranked by lane.  Ranks depend on no order of atomics: places are the stable sort's.  131072 slots take 12.7
// us on 16 SMs (scattered 4-byte stores), a decoding step's 264 on one CTA 2.2.
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
// WPR warps to a token's row, 8 warps to a CTA.  A thread takes words of WB bytes, the largest of 16, 4 and
// 2 that every row starts on, UC of them at a time from each of KC choices.  The choices' rows are
// looked up once for the whole row (MANY, k > 8: 8 at a time for each stretch of it): with a look-up by
// shuffles at each word the sums of 4093 x 4 rows of 1001 fp32 numbers took 40 us, issue 90 %.
constexpr int kRowWarps = 8;

template <int WB>
struct WordOf;
template <>
struct WordOf<16> { using type = uint4; };
template <>
struct WordOf<4> { using type = uint32_t; };
template <>
struct WordOf<2> { using type = uint16_t; };
template <int WB>
using Word = typename WordOf<WB>::type;

template <typename T, int WB>
constexpr int kNumbers = WB / static_cast<int>(sizeof(T));

template <typename T, int WB>
__device__ __forceinline__ void numbers(const Word<WB>& q, float (&v)[kNumbers<T, WB>]) {
    if constexpr (WB == 16) {
        unpack16(q, v);
    } else if constexpr (sizeof(T) == 4) {
        v[0] = __uint_as_float(q);
    } else {
        v[0] = __uint_as_float(static_cast<uint32_t>(q) << 16);
        if constexpr (WB == 4) v[1] = __uint_as_float(q & 0xFFFF0000u);
    }
}
template <typename T, int WB>
__device__ __forceinline__ Word<WB> word(const float (&v)[kNumbers<T, WB>]) {
    if constexpr (WB == 16) {
        return pack16(v);
    } else if constexpr (sizeof(T) == 4) {
        return __float_as_uint(v[0]);
    } else if constexpr (WB == 4) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        return __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    }
}
template <int WB>
__device__ __forceinline__ Word<WB> zero_word() {
    if constexpr (WB == 16) return make_uint4(0u, 0u, 0u, 0u);
    else return 0;
}

// Lane i's choice of a token: its place, -1 for none.
__device__ __forceinline__ int place_of(const int32_t* places, int64_t token, int k, int lane, int64_t rows) {
    if (lane >= k) return -1;
    const int at = places[token * k + lane];
    return at < rows ? at : -1;
}

// The rows of choices i0 .. i0 + KC - 1 in a buffer of rows; null for none.
template <typename T, int KC>
__device__ __forceinline__ void rows_of(T* base, int64_t stride, int place, int i0, T* (&row)[KC]) {
#pragma unroll
    for (int i = 0; i < KC; ++i) {
        const int at = __shfl_sync(kEvery, place, (i0 + i) & 31);
        row[i] = i0 + i < 32 && at >= 0 ? base + at * stride : nullptr;
    }
}

// The rows of a buffer behind the last choice, as many as slots are without an expert: zeros.
template <typename T, int WPR, int WB>
__device__ __forceinline__ void clear_behind(T* base, int64_t D, int n, int64_t filled, int64_t token, int k) {
    for (int64_t r = max(filled, token * k); r < (token + 1) * k; ++r) {
        Word<WB>* dst = reinterpret_cast<Word<WB>*>(base + r * D);
        for (int c = threadIdx.x % (WPR * 32); c < n; c += WPR * 32) dst[c] = zero_word<WB>();
    }
}

struct GatherParams {
    const void* x;
    const int32_t* places;
    const int32_t* offsets;
    void* out;
    int64_t tokens, stride;
    int32_t D, k, E;
};

template <typename T, int WPR, int WB, int KC, bool MANY>
__global__ void __launch_bounds__(kRowWarps * 32) ds_expert_gather_kernel(const GatherParams p) {
    constexpr int STEP = WPR * 32, UC = 4;
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t token = static_cast<int64_t>(blockIdx.x) * (kRowWarps / WPR) + threadIdx.x / STEP;
    if (token >= p.tokens) return;
    const int place = place_of(p.places, token, p.k, lane, p.tokens * p.k);
    const int64_t filled = p.offsets[p.E];
    const int n = p.D / kNumbers<T, WB>;
    const Word<WB>* src = reinterpret_cast<const Word<WB>*>(static_cast<const T*>(p.x) + token * p.stride);
    T* out = static_cast<T*>(p.out);
    T* row[KC];
    if (!MANY) rows_of(out, p.D, place, 0, row);
    for (int c0 = threadIdx.x % STEP - lane; c0 < n; c0 += STEP * UC) {  // the warp's words
        const int c = c0 + lane;
        Word<WB> v[UC];
#pragma unroll
        for (int u = 0; u < UC; ++u)
            if (c + u * STEP < n) v[u] = src[c + u * STEP];
        for (int i0 = 0; i0 < (MANY ? p.k : 1); i0 += KC) {
            if (MANY) rows_of(out, p.D, place, i0, row);
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                if (!row[i]) continue;
                Word<WB>* dst = reinterpret_cast<Word<WB>*>(row[i]) + c;
#pragma unroll
                for (int u = 0; u < UC; ++u)
                    if (c + u * STEP < n) dst[u * STEP] = v[u];
            }
        }
    }
    clear_behind<T, WPR, WB>(out, p.D, n, filled, token, p.k);
}

struct CombineParams {
    const void* y;
    const int32_t* places;
    const float* weights;
    void* out;
    int64_t tokens, rows, stride;
    int32_t D, k;
};

template <typename T, int WPR, int WB, int KC, bool MANY>
__global__ void __launch_bounds__(kRowWarps * 32) ds_expert_combine_kernel(const CombineParams p) {
    constexpr int STEP = WPR * 32, N = kNumbers<T, WB>, UC = WB == 16 ? (KC < 8 ? 2 : 1) : 4;
    const int lane = threadIdx.x & 31;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t token = static_cast<int64_t>(blockIdx.x) * (kRowWarps / WPR) + threadIdx.x / STEP;
    if (token >= p.tokens) return;
    const int place = place_of(p.places, token, p.k, lane, p.rows);
    const float weight = lane < p.k ? (p.weights ? p.weights[token * p.k + lane] : 1.f) : 0.f;
    const T* y = static_cast<const T*>(p.y);
    Word<WB>* out = reinterpret_cast<Word<WB>*>(static_cast<T*>(p.out) + token * p.D);
    const int n = p.D / N;
    const T* row[KC];
    float w[KC];
    const auto look_up = [&](int i0) {
        rows_of(y, p.stride, place, i0, row);
#pragma unroll
        for (int i = 0; i < KC; ++i) w[i] = __shfl_sync(kEvery, weight, (i0 + i) & 31);
    };
    if (!MANY) look_up(0);
    for (int c0 = threadIdx.x % STEP - lane; c0 < n; c0 += STEP * UC) {
        const int c = c0 + lane;
        float sum[UC][N] = {};
        for (int i0 = 0; i0 < (MANY ? p.k : 1); i0 += KC) {
            if (MANY) look_up(i0);
            Word<WB> v[KC][UC];
#pragma unroll
            for (int i = 0; i < KC; ++i)
#pragma unroll
                for (int u = 0; u < UC; ++u)
                    if (row[i] && c + u * STEP < n) v[i][u] = reinterpret_cast<const Word<WB>*>(row[i])[c + u * STEP];
#pragma unroll
            for (int i = 0; i < KC; ++i) {
                if (!row[i]) continue;  // what no choice holds has no part, whatever its weight
#pragma unroll
                for (int u = 0; u < UC; ++u) {
                    float f[N];
                    numbers<T, WB>(v[i][u], f);
#pragma unroll
                    for (int j = 0; j < N; ++j) sum[u][j] = fmaf(w[i], f[j], sum[u][j]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < UC; ++u)
            if (c + u * STEP < n) out[c + u * STEP] = word<T, WB>(sum[u]);
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

// KC choices at a time over the whole row (with more of them the gradient's row is read again, from L1): a
// lane sums its part of each choice's product, and the lanes' (and warps') parts are added in a fixed
// order.
template <typename T, int WPR, int WB, int KC>
__global__ void __launch_bounds__(kRowWarps * 32) ds_expert_combine_backward_kernel(const CombineBackParams p) {
    constexpr int STEP = WPR * 32, N = kNumbers<T, WB>, UC = WB == 16 ? 1 : 4;
    __shared__ float sh_part[kRowWarps][KC];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t token = static_cast<int64_t>(blockIdx.x) * (kRowWarps / WPR) + threadIdx.x / STEP;
    if (token >= p.tokens) return;  // (never one of a CTA that has a token to itself)
    const int place = place_of(p.places, token, p.k, lane, p.tokens * p.k);
    const int64_t filled = p.offsets[p.E];
    const float weight = lane < p.k ? p.weights[token * p.k + lane] : 0.f;
    const Word<WB>* g = reinterpret_cast<const Word<WB>*>(static_cast<const T*>(p.grad) + token * p.grad_stride);
    const int n = p.D / N;
    for (int i0 = 0; i0 < p.k; i0 += KC) {
        const T* row[KC];
        T* out[KC];
        float w[KC], dot[KC] = {};
        rows_of(static_cast<const T*>(p.y), p.stride, place, i0, row);
        rows_of(static_cast<T*>(p.grad_y), static_cast<int64_t>(p.D), place, i0, out);
#pragma unroll
        for (int i = 0; i < KC; ++i) w[i] = __shfl_sync(kEvery, weight, (i0 + i) & 31);
        for (int c = threadIdx.x % STEP; c < n; c += STEP * UC) {
            Word<WB> gw[UC], v[KC][UC];
#pragma unroll
            for (int u = 0; u < UC; ++u)
                if (c + u * STEP < n) gw[u] = g[c + u * STEP];
#pragma unroll
            for (int i = 0; i < KC; ++i)
#pragma unroll
                for (int u = 0; u < UC; ++u)
                    if (row[i] && c + u * STEP < n) v[i][u] = reinterpret_cast<const Word<WB>*>(row[i])[c + u * STEP];
#pragma unroll
            for (int u = 0; u < UC; ++u) {
                if (c + u * STEP >= n) break;
                float gv[N];
                numbers<T, WB>(gw[u], gv);
#pragma unroll
                for (int i = 0; i < KC; ++i) {
                    if (!row[i]) continue;
                    float yv[N], d[N];
                    numbers<T, WB>(v[i][u], yv);
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        dot[i] = fmaf(gv[j], yv[j], dot[i]);
                        d[j] = w[i] * gv[j];
                    }
                    reinterpret_cast<Word<WB>*>(out[i])[c + u * STEP] = word<T, WB>(d);
                }
            }
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
            mine = 0.f;
            if (warp == 0 && lane < KC)
                for (int v = 0; v < WPR; ++v) mine += sh_part[v][lane];
            __syncthreads();
        }
        if ((WPR == 1 || warp == 0) && lane < KC && i0 + lane < p.k) p.grad_weights[token * p.k + i0 + lane] = mine;
    }
    clear_behind<T, WPR, WB>(static_cast<T*>(p.grad_y), p.D, n, filled, token, p.k);
}

// ---------------------------------------------------------------- host --------------
// The bytes of a word that all rows of a buffer start on and D numbers are a multiple of.
static int word_bytes(const void* p, int64_t stride, int64_t D, int es) {
    const uint64_t all = reinterpret_cast<uintptr_t>(p) | static_cast<uint64_t>(stride * es) | static_cast<uint64_t>(D * es);
    return all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : 2;
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

template <typename T, int WB, int KC, bool MANY>
static ds_status launch_as(const GatherParams& p, int sms, cudaStream_t s) {
    return launch_rows(p, p.tokens, sms, s, ds_expert_gather_kernel<T, 1, WB, KC, MANY>, ds_expert_gather_kernel<T, 8, WB, KC, MANY>);
}
template <typename T, int WB, int KC, bool MANY>
static ds_status launch_as(const CombineParams& p, int sms, cudaStream_t s) {
    return launch_rows(p, p.tokens, sms, s, ds_expert_combine_kernel<T, 1, WB, KC, MANY>, ds_expert_combine_kernel<T, 8, WB, KC, MANY>);
}
template <typename T, int WB, int KC, bool MANY>
static ds_status launch_as(const CombineBackParams& p, int sms, cudaStream_t s) {
    return launch_rows(p, p.tokens, sms, s, ds_expert_combine_backward_kernel<T, 1, WB, KC>,
                       ds_expert_combine_backward_kernel<T, 8, WB, KC>);
}

template <typename T, int WB, typename P>
static ds_status launch_choices(const P& p, int sms, cudaStream_t s) {
    if (p.k <= 2) return launch_as<T, WB, 2, false>(p, sms, s);
    if (p.k <= 4) return launch_as<T, WB, 4, false>(p, sms, s);
    return p.k <= 8 ? launch_as<T, WB, 8, false>(p, sms, s) : launch_as<T, WB, 8, true>(p, sms, s);
}
template <typename P>
static ds_status launch_exchange(const P& p, int32_t dtype, int bytes, int sms, cudaStream_t s) {
    if (dtype == DS_FP32) return bytes == 16 ? launch_choices<float, 16>(p, sms, s) : launch_choices<float, 4>(p, sms, s);
    if (bytes == 16) return launch_choices<__nv_bfloat16, 16>(p, sms, s);
    return bytes == 4 ? launch_choices<__nv_bfloat16, 4>(p, sms, s) : launch_choices<__nv_bfloat16, 2>(p, sms, s);
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
    if (k > kMaxChoices || D > kMaxColumns || tokens > 0x7FFFFFFFLL / k) return DS_ERR_UNSUPPORTED;
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
    if (smem > 32768 &&  // (with the kernel's own arrays, past what needs no asking)
        cudaFuncSetAttribute(ds_expert_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSortWarps * kSortMaxE * static_cast<int>(sizeof(int32_t))) != cudaSuccess)
        return DS_ERR_CUDA;
    if (ctas > 8 && cudaFuncSetAttribute(ds_expert_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return DS_ERR_CUDA;
    // a thread for each expert, a warp for each that has slots
    const int threads = std::max((E + 31) / 32, std::max(p.warps, 1)) * 32;
    return launch_pdl(ds_expert_sort_kernel, dim3(ctas), threads, smem, ctas, stream, p);
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
    const int bytes = std::min(word_bytes(x, row_stride, D, es), word_bytes(out, D, D, es));
    int sms = 0;
    if (const ds_status st = device_sms(sms)) return st;
    return launch_exchange(p, dtype, bytes, sms, stream);
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
    const int bytes = std::min(word_bytes(y, row_stride, D, es), word_bytes(out, D, D, es));
    int sms = 0;
    if (const ds_status st = device_sms(sms)) return st;
    return launch_exchange(p, dtype, bytes, sms, stream);
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
    const int bytes = std::min({word_bytes(grad, grad_stride, D, es), word_bytes(y, row_stride, D, es), word_bytes(grad_y, D, D, es)});
    int sms = 0;
    if (const ds_status st = device_sms(sms)) return st;
    return launch_exchange(p, dtype, bytes, sms, stream);
}

}  // extern "C"
