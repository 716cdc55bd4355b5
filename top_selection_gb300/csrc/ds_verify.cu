// ds_verify.cu -- verification of drafted tokens against the target's probabilities.
//
// A sequence has S drafted tokens t_i and the target's logits x_i at S + 1 places (the last
// one follows the last draft).  With p_i = softmax(x_i / temperature) -- at temperature 0 the
// one-hot of the first maximum -- and q_i the distribution the draft was drawn from (one-hot
// at t_i where the draft has none), draft i is accepted iff every earlier one was and
//     u_i * q_i(t_i) < p_i(t_i).
// At the stop n (the first refused draft, or the place after the last) one more token is
// drawn from r = max(p_n - q_n, 0) after a refusal (from p_n where r is zero everywhere), else
// from p_n, as argmax_v r_v / e_v with e_v independent exponential draws: in such a race v
// wins with probability r_v / sum r, and no running sum over the vocabulary is needed.  The
// emitted tokens are then distributed as the target's own samples.
//
// One CTA per sequence takes the rows in order and stops at the refused one: a pass for the
// row's maximum and sum of exponentials, then one pass over the stop row, q_n and e.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kVerThreads = 1024;

struct VerifyParams {
    const void* logits;
    int64_t seq_stride, row_stride;  // elements
    const float* q;
    int64_t q_seq, q_row;
    const int32_t* drafts;
    const int32_t* lens;
    const float* uniforms;
    const float* noise;
    int64_t noise_stride;
    const float* temps;
    float temperature;
    int32_t S, V;
    int32_t* tokens;
    int32_t* accepted;
    float* probs;
};

__device__ __forceinline__ float ver_f32(float v) { return v; }
__device__ __forceinline__ float ver_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// The larger (value, lower index) of two candidates.
__device__ __forceinline__ void best_of(float& v, int& i, float v2, int i2) {
    if (v2 > v || (v2 == v && i2 < i)) {
        v = v2;
        i = i2;
    }
}

// exp((x - max) / temperature), 0 for -inf and for a row of -inf alone
__device__ __forceinline__ float weight(float x, float mx, float inv_t) {
    return x == -INFINITY ? 0.f : expf((x - mx) * inv_t);
}

template <typename T>
__global__ void __launch_bounds__(kVerThreads) ds_verify_kernel(const VerifyParams p) {
    __shared__ float sh_a[32], sh_b[32];
    __shared__ int sh_i[32], sh_j[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t b = blockIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    const float temp = p.temps ? p.temps[b] : p.temperature;
    const bool greedy = !(temp > 0.f);
    const float inv_t = greedy ? 1.f : 1.f / temp;
    const int len = p.lens ? min(max(p.lens[b], 0), p.S) : p.S;
    int32_t* tokens = p.tokens + b * (p.S + 1);
    float* probs = p.probs ? p.probs + b * (p.S + 1) : nullptr;
    int n = 0;
    for (;; ++n) {
        const T* x = static_cast<const T*>(p.logits) + b * p.seq_stride + n * p.row_stride;
        // the row's first maximum, and the sum of exponentials
        float mx = -INFINITY;
        int at = 0x7FFFFFFF;
        for (int v = tid; v < p.V; v += kVerThreads) best_of(mx, at, ver_f32(x[v]), v);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1)
            best_of(mx, at, __shfl_xor_sync(0xFFFFFFFFu, mx, d), __shfl_xor_sync(0xFFFFFFFFu, at, d));
        if (lane == 0) sh_a[warp] = mx, sh_i[warp] = at;
        __syncthreads();
        mx = sh_a[lane], at = sh_i[lane];
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1)
            best_of(mx, at, __shfl_xor_sync(0xFFFFFFFFu, mx, d), __shfl_xor_sync(0xFFFFFFFFu, at, d));
        float sum = 0.f;
        if (!greedy) {
            for (int v = tid; v < p.V; v += kVerThreads) sum += weight(ver_f32(x[v]), mx, inv_t);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
            if (lane == 0) sh_b[warp] = sum;
            __syncthreads();
            sum = sh_b[lane];
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        }
        const auto prob = [&](int v, float xv) {
            if (mx == -INFINITY) return 0.f;
            return greedy ? (v == at ? 1.f : 0.f) : weight(xv, mx, inv_t) / sum;
        };
        const bool drafted = n < len;
        int t = -1;
        float qt = 1.f;
        const float* q = nullptr;
        if (drafted) {
            t = p.drafts[b * p.S + n];
            if (t < 0 || t >= p.V) t = -1;  // no column: refused
            if (p.q) {
                q = p.q + b * p.q_seq + n * p.q_row;
                if (t >= 0) qt = q[t];
            }
            const float pt = t >= 0 ? prob(t, ver_f32(x[t])) : 0.f;
            if (p.uniforms[b * p.S + n] * qt < pt) {
                if (tid == 0) {
                    tokens[n] = t;
                    if (probs) probs[n] = pt;
                }
                __syncthreads();
                continue;
            }
        }
        // the stop row: the best of r / e, and of p / e should r be zero everywhere
        const float* noise = p.noise + b * p.noise_stride;
        float r1 = 0.f, r2 = 0.f;
        int i1 = 0x7FFFFFFF, i2 = 0x7FFFFFFF;
        for (int v = tid; v < p.V; v += kVerThreads) {
            const float pv = prob(v, ver_f32(x[v])), e = noise[v];
            const float qv = !drafted ? 0.f : q ? q[v] : v == t ? 1.f : 0.f;
            const float r = fmaxf(pv - qv, 0.f);
            if (r > 0.f) best_of(r1, i1, r / e, v);
            if (pv > 0.f) best_of(r2, i2, pv / e, v);
        }
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) {
            best_of(r1, i1, __shfl_xor_sync(0xFFFFFFFFu, r1, d), __shfl_xor_sync(0xFFFFFFFFu, i1, d));
            best_of(r2, i2, __shfl_xor_sync(0xFFFFFFFFu, r2, d), __shfl_xor_sync(0xFFFFFFFFu, i2, d));
        }
        __syncthreads();
        if (lane == 0) sh_a[warp] = r1, sh_i[warp] = i1, sh_b[warp] = r2, sh_j[warp] = i2;
        __syncthreads();
        if (warp == 0) {
            r1 = sh_a[lane], i1 = sh_i[lane], r2 = sh_b[lane], i2 = sh_j[lane];
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) {
                best_of(r1, i1, __shfl_xor_sync(0xFFFFFFFFu, r1, d), __shfl_xor_sync(0xFFFFFFFFu, i1, d));
                best_of(r2, i2, __shfl_xor_sync(0xFFFFFFFFu, r2, d), __shfl_xor_sync(0xFFFFFFFFu, i2, d));
            }
            const int last = i1 < p.V ? i1 : i2 < p.V ? i2 : -1;  // -1: the row has no distribution
            const float pl = last >= 0 ? prob(last, ver_f32(x[last])) : 0.f;
            for (int i = n + lane; i <= p.S; i += 32) {
                tokens[i] = i == n ? last : -1;
                if (probs) probs[i] = i == n ? pl : 0.f;
            }
            if (lane == 0) p.accepted[b] = n;
        }
        return;
    }
}

}  // namespace dsk

using namespace dsk;

extern "C" {

ds_status ds_verify_drafts(const void* logits, int32_t dtype, int64_t sequences, int32_t drafts_per_sequence,
                           int64_t V, int64_t seq_stride, int64_t row_stride, const int32_t* drafts,
                           const int32_t* draft_lens, const float* draft_probs, int64_t probs_seq_stride,
                           int64_t probs_row_stride, const float* uniforms, const float* noise, int64_t noise_stride,
                           const float* temperatures, float temperature, int32_t* out_tokens, int32_t* out_accepted,
                           float* out_probs, cudaStream_t stream) {
    const int32_t S = drafts_per_sequence;
    if ((dtype != DS_BF16 && dtype != DS_FP32) || sequences < 0 || S < 0 || V < 1) return DS_ERR_INVALID_ARG;
    if (row_stride < V || noise_stride < V || seq_stride < 0) return DS_ERR_INVALID_ARG;
    if (draft_probs && S > 0 && (probs_row_stride < V || probs_seq_stride < 0)) return DS_ERR_INVALID_ARG;
    if (!temperatures && !(temperature >= 0.f && temperature < INFINITY)) return DS_ERR_INVALID_ARG;
    if (V > (int64_t(1) << 30) || S > 1024 || sequences > 0x7FFFFFFFLL) return DS_ERR_UNSUPPORTED;
    if (sequences == 0) return DS_OK;
    if (!logits || !noise || !out_tokens || !out_accepted || (S > 0 && (!drafts || !uniforms)))
        return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    const void* words[] = {drafts, draft_lens, draft_probs, uniforms, noise, temperatures, out_tokens, out_accepted, out_probs};
    for (const void* w : words)
        if (reinterpret_cast<uintptr_t>(w) % 4) return DS_ERR_ALIGNMENT;
    if (reinterpret_cast<uintptr_t>(logits) % es) return DS_ERR_ALIGNMENT;
    const VerifyParams p = {logits, seq_stride, row_stride, draft_probs, probs_seq_stride, probs_row_stride, drafts,
                            draft_lens, uniforms, noise, noise_stride, temperatures, temperature, S,
                            static_cast<int32_t>(V), out_tokens, out_accepted, out_probs};
    const dim3 grid(static_cast<unsigned>(sequences));
    return dtype == DS_BF16 ? launch_pdl(ds_verify_kernel<__nv_bfloat16>, grid, kVerThreads, 0, 1, stream, p)
                            : launch_pdl(ds_verify_kernel<float>, grid, kVerThreads, 0, 1, stream, p);
}

}  // extern "C"
