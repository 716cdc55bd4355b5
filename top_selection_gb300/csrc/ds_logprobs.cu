// ds_logprobs.cu -- log probabilities of given tokens with the distribution's entropy and its
// likeliest tokens (ds_token_logprobs), and their gradient (ds_token_logprobs_backward).
//
// For a row x of V logits, m its largest, s = sum exp(x - m), w = sum exp(x - m) (x - m):
//   lse = m + log s,   log p_v = (x_v - m) - log s,   H = -sum p log p = log s - w / s
// and with gradients g of the given token's log p_t and h of H:
//   dx_v = g ([v = t] - p_v) - h p_v (log p_v + H).
// One pass over the row: a thread keeps m, s and w of what it has seen (rescaled when its m rises),
// 32 numbers at a time in registers.  The `top` largest are found in the same pass: a threshold
// that at least `top` numbers reach, from the maxima of groups of threads over the first 32
// numbers each, then what lies above it goes to a short list, cut back to its `top` largest (which
// raises the threshold) when it has grown.  Order is by value, then by the lower index, so keys are
// 64 bits (order-preserving value, inverted index) and distinct.  A row's parts on the CTAs of a
// cluster are joined by the first, over distributed shared memory, in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_rows.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kLogThreads = 256;
constexpr int kLogWarps = kLogThreads / 32;
constexpr int kLogCluster = 16;      // most CTAs to a row
constexpr int kLogMaxTop = 32;
constexpr int kLogGroups = 64;       // groups of threads whose maxima give the first threshold
constexpr int kLogList = 512;        // places of a CTA's list (and of the join: 16 x 32)
constexpr int kLogRoom = 128;        // a list this much over `top` is cut back
constexpr int kLogHeld = 32;         // numbers a thread holds at a time
constexpr uint32_t kLanes = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 2^x within 2^-22; 0 below 2^-126.
__device__ __forceinline__ float exp2_term(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

struct LogParams {
    const void* x;
    const int32_t* tokens;
    float* logprobs;
    float* lse;
    float* entropy;
    float* top_logprobs;
    int32_t* top_tokens;
    int64_t rows, stride;
    int32_t V, top;
    int32_t per_cta;  // 16-byte words of a row to a CTA
};

// m, s, w of a part of a row, w in units of ln 2: sums of 2^y and 2^y y with y = (x - m) log2 e.
struct Part {
    float m, s, w;
};
__device__ __forceinline__ void rise(Part& a, float m) {  // to a larger m
    if (m > a.m) {
        if (a.s > 0.f) {
            const float d = fmaxf((a.m - m) * kLog2e, -150.f), f = exp2_term(d);
            a.w = f * fmaf(a.s, d, a.w);
            a.s *= f;
        }
        a.m = m;
    }
}
__device__ __forceinline__ void join(Part& a, Part b) {
    const float m = fmaxf(a.m, b.m);
    rise(a, m);
    rise(b, m);
    a.s += b.s;
    a.w += b.w;
}

// 16 bytes of the row, word g of it counted from the 16-byte boundary at or below its start
// (`shift` numbers before it); numbers outside the row are -inf.
template <typename T>
__device__ __forceinline__ uint4 row_word(const T* row, int g, int shift, int V) {
    constexpr int PER = kPer<T>;
    const int at = g * PER - shift;
    if (at >= 0 && at + PER <= V) return *reinterpret_cast<const uint4*>(row + at);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            w[i] = at + i >= 0 && at + i < V ? __float_as_uint(row[at + i]) : 0xFF800000u;
        } else {
            const int a = at + 2 * i;
            const uint32_t lo = a >= 0 && a < V ? reinterpret_cast<const uint16_t*>(row)[a] : 0xFF80u;
            const uint32_t hi = a + 1 >= 0 && a + 1 < V ? reinterpret_cast<const uint16_t*>(row)[a + 1] : 0xFF80u;
            w[i] = lo | hi << 16;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ uint4 no_word() {
    const uint32_t f = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
    return make_uint4(f, f, f, f);
}

// The largest of a word's numbers.
template <typename T>
__device__ __forceinline__ float word_max(const uint4& q) {
    if constexpr (sizeof(T) == 4) {
        return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
    } else {
        const auto pair = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
        const __nv_bfloat162 m = __hmax2(__hmax2(pair(q.x), pair(q.y)), __hmax2(pair(q.z), pair(q.w)));
        return fmaxf(__low2float(m), __high2float(m));
    }
}

__device__ __forceinline__ uint64_t order_key(float v, int at) {
    return static_cast<uint64_t>(key_f32(__float_as_uint(v + 0.f))) << 32 | static_cast<uint32_t>(~at);  // -0 equals +0
}
__device__ __forceinline__ float key_value(uint64_t k) { return __uint_as_float(unkey_f32(static_cast<uint32_t>(k >> 32))); }
__device__ __forceinline__ int key_at(uint64_t k) { return static_cast<int>(~static_cast<uint32_t>(k)); }

struct LogShared {
    uint64_t list[kLogList];
    uint64_t best[kLogMaxTop];  // the largest so far, in order
    float group[kLogGroups];
    uint64_t reduce[kLogWarps];
    Part parts[kLogWarps];
    Part part;                  // the CTA's
    float edge;
    int count, kept;
};

// The `top` largest of list[0 .. count), in order, to best[]: each entry's rank is the number of
// larger ones.  Called by all threads; list and count are complete, best is afterwards.
__device__ __forceinline__ void cut_list(LogShared& sh, int count, int top) {
    for (int i = threadIdx.x; i < count; i += kLogThreads) {
        const uint64_t k = sh.list[i];
        int above = 0;
        for (int j = 0; j < count; ++j) above += sh.list[j] > k ? 1 : 0;
        if (above < top) sh.best[above] = k;
    }
    if (threadIdx.x == 0) sh.kept = min(count, top);
    __syncthreads();
}

template <typename T, bool TOP>
__global__ void __launch_bounds__(kLogThreads, 4) ds_token_logprobs_kernel(const LogParams p) {
    constexpr int PER = kPer<T>, U = kLogHeld / PER;
    __shared__ LogShared sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ctas = gridDim.x, rank = blockIdx.x;  // of the row
    const int64_t row = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
    pdl_launch_dependents();
    if (row >= p.rows) return;  // a whole cluster
    if (TOP && tid == 0) sh.count = sh.kept = 0;
    const T* x = static_cast<const T*>(p.x) + row * p.stride;
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
    const int words = (p.V + shift + PER - 1) / PER;
    const int first = min(words, static_cast<int>(rank) * p.per_cta), last = min(words, first + p.per_cta);
    if (TOP) __syncthreads();
    pdl_wait();

    Part a = {-INFINITY, 0.f, 0.f};
    float edge = -INFINITY;  // at least `top` numbers of earlier chunks reach it (or it is -inf)
    for (int g0 = first; g0 < last; g0 += kLogThreads * U) {
        uint4 q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = g0 + u * kLogThreads + tid;
            q[u] = g < last ? row_word(x, g, shift, p.V) : no_word<T>();
        }
        float most = word_max<T>(q[0]);
#pragma unroll
        for (int u = 1; u < U; ++u) most = fmaxf(most, word_max<T>(q[u]));
        rise(a, most);
        const float m = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[PER];
            unpack16(q[u], v);
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const float y = fmaxf((v[j] - m) * kLog2e, -150.f), e = exp2_term(y);
                a.s += e;
                a.w = fmaf(e, y, a.w);
            }
        }
        if constexpr (TOP) {
            // a way of finding what may be among the largest: 0, numbers above the edge so far (their
            // indices are all higher, so equal ones lose); 1, an edge from this chunk as well, which
            // equal numbers reach; 2, in turn, one number at a time, where thousands are equal
            bool fits = false;
            int count = 0;
            for (int way = g0 == first ? 1 : 0; way < 2 && !fits; ++way) {
                float e = edge;
                if (way == 1) {
                    const float g = lanes_max<4>(most);
                    if (lane % 4 == 0) sh.group[tid / 4] = g;
                    if (tid == 0) sh.count = sh.kept;
                    __syncthreads();
                    if (warp == 0) {  // the largest group maximum that `top` of them reach
                        const float g0v = sh.group[lane], g1v = sh.group[lane + 32];
                        int n0 = 0, n1 = 0;
#pragma unroll 8
                        for (int j = 0; j < kLogGroups; ++j) {
                            const float o = sh.group[j];
                            n0 += o >= g0v ? 1 : 0;
                            n1 += o >= g1v ? 1 : 0;
                        }
                        const float c = lanes_max<32>(fmaxf(n0 >= p.top ? g0v : -INFINITY, n1 >= p.top ? g1v : -INFINITY));
                        if (lane == 0) sh.edge = c;
                    }
                    __syncthreads();
                    e = fmaxf(edge, sh.edge);
                }
                // numbers at the edge of earlier chunks lose to those, at this chunk's they may win
                const bool equal = e > edge;
                if (equal ? most >= e : most > e) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        const float wm = word_max<T>(q[u]);
                        if (!(equal ? wm >= e : wm > e)) continue;
                        float v[PER];
                        unpack16(q[u], v);
                        const int at = (g0 + u * kLogThreads + tid) * PER - shift;
#pragma unroll
                        for (int j = 0; j < PER; ++j)
                            if (equal ? v[j] >= e : v[j] > e) {
                                const int n = atomicAdd(&sh.count, 1);
                                if (n < kLogList) sh.list[n] = order_key(v[j], at + j);
                            }
                    }
                }
                __syncthreads();
                count = sh.count;
                fits = count <= kLogList;
                __syncthreads();  // the next append comes after everyone's look at the count
            }
            if (!fits) {
                uint64_t below = ~0ull;
                int found = sh.kept;
                for (int i = 0; i < p.top; ++i) {
                    uint64_t k = 0;
#pragma unroll 1
                    for (int u = 0; u < U; ++u) {  // (read again: rare, and the registers are dear)
                        const int g = g0 + u * kLogThreads + tid, at = g * PER - shift;
                        float v[PER];
                        unpack16(g < last ? row_word(x, g, shift, p.V) : no_word<T>(), v);
#pragma unroll
                        for (int j = 0; j < PER; ++j) {
                            const uint64_t c = v[j] > edge ? order_key(v[j], at + j) : 0;
                            k = c < below && c > k ? c : k;
                        }
                    }
#pragma unroll
                    for (int d = 16; d >= 1; d >>= 1) {
                        const uint64_t o = __shfl_xor_sync(kLanes, k, d);
                        k = o > k ? o : k;
                    }
                    if (lane == 0) sh.reduce[warp] = k;
                    __syncthreads();
                    k = 0;
                    for (int w = 0; w < kLogWarps; ++w) k = sh.reduce[w] > k ? sh.reduce[w] : k;
                    __syncthreads();
                    if (k == 0) break;
                    if (tid == 0) sh.list[found] = k;
                    ++found;
                    below = k;
                }
                if (tid == 0) sh.count = found;
                count = found;
                __syncthreads();
            }
            if (g0 + kLogThreads * U >= last || g0 == first || count > p.top + kLogRoom) {
                cut_list(sh, count, p.top);
                if (tid < sh.kept) sh.list[tid] = sh.best[tid];
                if (tid == 0) sh.count = sh.kept;
                if (sh.kept == p.top) edge = key_value(sh.best[p.top - 1]);
                __syncthreads();
            } else if (tid == 0) {
                sh.kept = count;  // entries that a second way starts behind
            }
        }
    }

    // the CTA's part, in the order of its warps
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        const Part b = {__shfl_xor_sync(kLanes, a.m, d), __shfl_xor_sync(kLanes, a.s, d), __shfl_xor_sync(kLanes, a.w, d)};
        // the same order of additions in both lanes of a pair
        Part lo = (lane & d) ? b : a;
        join(lo, (lane & d) ? a : b);
        a = lo;
    }
    if (lane == 0) sh.parts[warp] = a;
    __syncthreads();
    if (tid == 0) {
        Part c = sh.parts[0];
        for (int w = 1; w < kLogWarps; ++w) join(c, sh.parts[w]);
        sh.part = c;
    }
    if (ctas > 1) {
        cluster_sync_all();
        if (rank == 0) {
            if (tid == 0) {
                Part c = sh.part;
                for (uint32_t r = 1; r < ctas; ++r) {
                    const uint32_t from = map_rank(&sh.part, r);
                    join(c, {__uint_as_float(ld_cluster_u32(from)), __uint_as_float(ld_cluster_u32(from + 4)),
                             __uint_as_float(ld_cluster_u32(from + 8))});
                }
                sh.parts[0] = c;  // (part itself stays as it is for nobody: only rank 0 reads)
            }
            if constexpr (TOP) {
                // best[] of every CTA behind one another; places without an entry get keys below all
                for (int i = tid; i < static_cast<int>(ctas) * p.top; i += kLogThreads) {
                    const uint32_t r = i / p.top, j = i % p.top;
                    const int kept = static_cast<int>(ld_cluster_u32(map_rank(&sh.kept, r)));
                    uint64_t k = static_cast<uint64_t>(i);  // distinct, and below every number's key
                    if (static_cast<int>(j) < kept) {
                        const uint32_t from = map_rank(&sh.best[j], r);
                        k = static_cast<uint64_t>(ld_cluster_u32(from + 4)) << 32 | ld_cluster_u32(from);
                    }
                    sh.list[i] = k;
                }
            }
        }
        cluster_sync_all();
        if (rank != 0) return;
        if constexpr (TOP) cut_list(sh, static_cast<int>(ctas) * p.top, p.top);
    } else {
        if (tid == 0) sh.parts[0] = sh.part;
    }
    __syncthreads();
    const Part all = sh.parts[0];
    const float logs = all.s > 0.f ? logf(all.s) : 0.f;
    const auto log_p = [&](float v) { return all.s > 0.f ? (v - all.m) - logs : -INFINITY; };
    if (tid == 0) {
        const int t = p.tokens[row];
        p.logprobs[row] = t >= 0 && t < p.V ? log_p(row_f32(x[t])) : 0.f;
        p.lse[row] = all.m + logs;
        p.entropy[row] = all.s > 0.f ? fmaxf(logs - all.w * kLn2 / all.s, 0.f) : 0.f;
    }
    if constexpr (TOP) {
        if (warp != 0) return;
        const uint64_t k = lane < p.top ? sh.best[lane] : 0;
        bool real = lane < p.top && lane < sh.kept && (k >> 32) > 0x007FFFFFu;  // above -inf's key
        float v = real ? key_value(k) : -INFINITY;
        int at = real ? key_at(k) : 0;
        // fewer numbers above -inf than asked for: the first of the others follow
        int have = __popc(__ballot_sync(kLanes, real));
        for (int i0 = 0; have < p.top && i0 < p.V; i0 += 32) {
            const bool other = i0 + lane < p.V && !(row_f32(x[i0 + lane]) > -INFINITY);
            const uint32_t which = __ballot_sync(kLanes, other);
            const int n = __popc(which);
            if (lane >= have && lane < have + n) at = i0 + static_cast<int>(__fns(which, 0, lane - have + 1));
            have += n;
        }
        if (lane < p.top) {
            p.top_logprobs[row * p.top + lane] = log_p(v);
            p.top_tokens[row * p.top + lane] = at;
        }
    }
}

// ---------------------------------------------------------------- gradient ----------
// One number in, one out; a CTA takes a run of one row.  lse is rounded to fp32 (2^-24 of its size),
// which moves every p of the row by that much of itself.
constexpr int kBackThreads = 256;

struct LogBackParams {
    const void* x;
    const int32_t* tokens;
    const float* grad;
    const float* lse;
    const float* grad_entropy;
    const float* entropy;
    void* out;
    int64_t rows, stride, out_stride;
    int32_t V;
    int32_t runs;  // CTAs to a row
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(kBackThreads) ds_token_logprobs_backward_kernel(const LogBackParams p) {
    constexpr int PER = kPer<T>, U = 4;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x / p.runs;
    const int run = static_cast<int>(blockIdx.x % p.runs);
    const T* x = static_cast<const T*>(p.x) + row * p.stride;
    T* out = static_cast<T*>(p.out) + row * p.out_stride;
    int t = p.tokens[row];
    const float lse = p.lse[row];
    float g = p.grad[row], h = 0.f, H = 0.f;
    if (p.grad_entropy) h = p.grad_entropy[row], H = p.entropy[row];
    if (t < 0 || t >= p.V) t = -1, g = 0.f;
    const bool none = lse == -INFINITY;  // a row of -inf alone has no probabilities: no gradient
    const float z = none ? 0.f : lse;
    // -p (g + h (log p + H)), with log p bounded so that 0 times it stays 0
    const auto grad_of = [&](float v) {
        const float lp = fmaxf(v - z, -150.f);
        return -exp2_term(lp * kLog2e) * fmaf(h, lp + H, g);
    };
    if (VEC) {
        // both rows lie alike against 16-byte boundaries
        const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
        const int words = (p.V + shift + PER - 1) / PER, w0 = run * (kBackThreads * U);
        uint4 q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int w = w0 + u * kBackThreads + threadIdx.x;
            q[u] = w < words ? row_word(x, w, shift, p.V) : no_word<T>();
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int w = w0 + u * kBackThreads + threadIdx.x, at = w * PER - shift;
            if (w >= words) break;
            float v[PER];
            unpack16(q[u], v);
#pragma unroll
            for (int j = 0; j < PER; ++j) v[j] = none ? 0.f : grad_of(v[j]);
            if (!none && t >= at && t < at + PER) {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (at + j == t) v[j] += g;
            }
            if (at >= 0 && at + PER <= p.V) {
                *reinterpret_cast<uint4*>(out + at) = pack16(v);
            } else {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (at + j >= 0 && at + j < p.V) row_put(out + at + j, v[j]);
            }
        }
    } else {
        const int64_t c0 = static_cast<int64_t>(run) * (kBackThreads * U * PER);
#pragma unroll 8
        for (int i = 0; i < U * PER; ++i) {
            const int64_t c = c0 + i * kBackThreads + threadIdx.x;
            if (c < p.V) row_put(out + c, none ? 0.f : grad_of(row_f32(x[c])) + (c == t ? g : 0.f));
        }
    }
}

// ---------------------------------------------------------------- host --------------
template <typename T>
static ds_status launch_logprobs(LogParams p, int sms, cudaStream_t stream) {
    // a CTA to a row where rows are many; else as many as give every SM two, of 32 numbers a thread
    // at least
    constexpr int PER = kPer<T>, CHUNK = kLogThreads * kLogHeld;
    const int64_t words = (static_cast<int64_t>(p.V) + 2 * PER - 2) / PER;
    int ctas = 1;
    while (ctas < kLogCluster && p.rows * ctas < 2 * sms && static_cast<int64_t>(ctas) * CHUNK < p.V) ctas *= 2;
    p.per_cta = static_cast<int32_t>((words + ctas - 1) / ctas);
    const unsigned y = static_cast<unsigned>(p.rows < 65535 ? p.rows : 65535);
    const dim3 grid(ctas, y, static_cast<unsigned>((p.rows + y - 1) / y));
    const auto kern = p.top > 0 ? ds_token_logprobs_kernel<T, true> : ds_token_logprobs_kernel<T, false>;
    if (ctas > 8 && cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return DS_ERR_CUDA;
    return launch_pdl(kern, grid, kLogThreads, 0, ctas, stream, p);
}

static bool misaligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes != 0; }

}  // namespace dsk

using namespace dsk;

extern "C" {

ds_status ds_token_logprobs(const void* logits, int32_t dtype, int64_t rows, int64_t V, int64_t row_stride,
                            const int32_t* tokens, int32_t top, float* out_logprobs, float* out_lse, float* out_entropy,
                            float* out_top_logprobs, int32_t* out_top_tokens, cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || rows < 0 || V < 1 || row_stride < V || top < 0 || top > V)
        return DS_ERR_INVALID_ARG;
    if (top > kLogMaxTop || V > (1LL << 30) || rows > 0x7FFFFFFFLL) return DS_ERR_UNSUPPORTED;
    if (rows == 0) return DS_OK;
    if (!logits || !tokens || !out_logprobs || !out_lse || !out_entropy) return DS_ERR_INVALID_ARG;
    if (top > 0 && (!out_top_logprobs || !out_top_tokens)) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    if (misaligned(logits, es) || misaligned(tokens, 4) || misaligned(out_logprobs, 4) || misaligned(out_lse, 4) ||
        misaligned(out_entropy, 4) || misaligned(out_top_logprobs, 4) || misaligned(out_top_tokens, 4))
        return DS_ERR_ALIGNMENT;
    int dev = 0;
    DevInfo info;
    if (cudaGetDevice(&dev) != cudaSuccess || !dev_info(dev, info)) return DS_ERR_CUDA;
    const LogParams p = {logits, tokens, out_logprobs, out_lse, out_entropy, out_top_logprobs, out_top_tokens,
                         rows, row_stride, static_cast<int32_t>(V), top, 0};
    return dtype == DS_BF16 ? launch_logprobs<__nv_bfloat16>(p, info.sms, stream) : launch_logprobs<float>(p, info.sms, stream);
}

ds_status ds_token_logprobs_backward(const float* grad_logprobs, const void* logits, int32_t dtype, int64_t rows,
                                     int64_t V, int64_t row_stride, const int32_t* tokens, const float* lse,
                                     const float* grad_entropy, const float* entropy, void* grad_logits,
                                     int64_t grad_stride, cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || rows < 0 || V < 1 || row_stride < V || grad_stride < V)
        return DS_ERR_INVALID_ARG;
    if (V > (1LL << 30) || rows > 0x7FFFFFFFLL) return DS_ERR_UNSUPPORTED;
    if (rows == 0) return DS_OK;
    if (!grad_logprobs || !logits || !tokens || !lse || !grad_logits || (grad_entropy && !entropy)) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    if (misaligned(logits, es) || misaligned(grad_logits, es) || misaligned(tokens, 4) || misaligned(grad_logprobs, 4) ||
        misaligned(lse, 4) || misaligned(grad_entropy, 4) || misaligned(entropy, 4))
        return DS_ERR_ALIGNMENT;
    const int64_t per = 16 / es, words = (V + 2 * per - 2) / per, runs = (words + kBackThreads * 4 - 1) / (kBackThreads * 4);
    if (rows > 0x7FFFFFFFLL / runs) return DS_ERR_UNSUPPORTED;
    const LogBackParams p = {logits, tokens, grad_logprobs, lse, grad_entropy, entropy, grad_logits, rows, row_stride,
                             grad_stride, static_cast<int32_t>(V), static_cast<int32_t>(runs)};
    // 16 bytes at a time where a row and its gradient start at the same place of such a word
    const bool vec = (reinterpret_cast<uintptr_t>(logits) - reinterpret_cast<uintptr_t>(grad_logits)) % 16 == 0 &&
                     (rows == 1 || (row_stride - grad_stride) * es % 16 == 0);
    const dim3 grid(static_cast<unsigned>(rows * runs));
    const auto go = [&](auto kern) { return launch_pdl(kern, grid, kBackThreads, 0, 1, stream, p); };
    if (dtype == DS_BF16)
        return vec ? go(ds_token_logprobs_backward_kernel<__nv_bfloat16, true>) : go(ds_token_logprobs_backward_kernel<__nv_bfloat16, false>);
    return vec ? go(ds_token_logprobs_backward_kernel<float, true>) : go(ds_token_logprobs_backward_kernel<float, false>);
}

}  // extern "C"
