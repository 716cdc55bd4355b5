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
// numbers each; then 16-byte words with a number above it go to a list as they are, which is cut back to its
// `top` largest numbers (and raises the threshold) after 2, 8, 32 .. chunks and at the end.  Order is by
// value, NaN first, then by the lower index, so keys are 64 bits (order-preserving value, inverted index) and
// distinct.  A row's parts on the CTAs of a cluster are joined by the first, over distributed shared
// memory, in a fixed order.
//
// Long rows are bound by memory (2048 x 129280 bf16: 89 us, 88 % of the copy rate; the gradient 153 us for
// reading and writing it, the copy rate), short ones by their starts and barriers (4099 x 32003 bf16: 49 us, 79 %),
// and the top by the cuts' barriers and single steps: 66 us with one token, 88 with 20 (numbers listed one
// by one: 126).  One row of 129280 fp32 numbers on 16 CTAs takes 2.7 us, with 20 tokens 7.9.  Terms from one fma,
// x log2 e - m log2 e, took 1 % less of the rows with a top, and lost all digits of rows of large logits.  Tried and not kept:
// rings of bulk copies in shared memory (registers for 20 warps an SM: 84 us with one token), a warp to a row (73),
// one warp that cuts while the others go on (85), CTAs that take rows in turn with the next row's first words on
// their way (77).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_rows.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kLogThreads = 256, kLogFewThreads = 128;  // of a CTA: a cluster's, a row's own
constexpr int kLogCluster = 16;      // most CTAs to a row
constexpr int kLogMaxTop = 32;
constexpr int kLogGroups = 64;       // groups of threads whose maxima give the first threshold
constexpr int kLogHits = 256;        // words of a CTA's list of those with a number above the edge
constexpr int kLogFew = 48;          // that are cut without looking for a higher edge first
constexpr int kLogList = 512;        // numbers to be ranked (and a half of the join's lists, 16 x 32)
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

// Sums over a part of a row whose largest number is m: s of 2^y and w of 2^y y, with y = (x - m) log2 e.  The
// difference comes first: it is exact where x lies within a factor of two of m, so that a term is off by
// roundings of y alone, whatever the size of m.
struct Part {
    float m, s, w;
};

// Differences of larger numbers may leave fp32's range.  fp32's steps are 10^30 there: beside a part's largest
// number of that size only its equals count.
constexpr float kFar = 1e37f;
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) > kFar; }

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
using Two = unsigned long long;  // two fp32 numbers, for the packed instructions
__device__ __forceinline__ Two two(float a, float b) {
    return static_cast<Two>(__float_as_uint(b)) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ float lower(Two a) { return __uint_as_float(static_cast<uint32_t>(a)); }
__device__ __forceinline__ float upper(Two a) { return __uint_as_float(static_cast<uint32_t>(a >> 32)); }
__device__ __forceinline__ Two fma_two(Two a, Two b, Two c) {
    Two d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ Two mul_two(Two a, Two b) {
    Two d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ Two add_two(Two a, Two b) {
    Two d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
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

// The larger number, NaN where one of them is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// The largest of a word's numbers, NaN where one of them is.
template <typename T>
__device__ __forceinline__ float word_max_or_nan(const uint4& q) {
    if constexpr (sizeof(T) == 4) {
        return max_or_nan(max_or_nan(__uint_as_float(q.x), __uint_as_float(q.y)),
                          max_or_nan(__uint_as_float(q.z), __uint_as_float(q.w)));
    } else {
        const auto pair = [](uint32_t u) { return *reinterpret_cast<const __nv_bfloat162*>(&u); };
        const __nv_bfloat162 m = __hmax2_nan(__hmax2_nan(pair(q.x), pair(q.y)), __hmax2_nan(pair(q.z), pair(q.w)));
        return max_or_nan(__low2float(m), __high2float(m));
    }
}

// The largest of a word's numbers, NaN left out.
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

// the two halves of a cluster barrier: the arrivals tell that the CTAs run
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_cluster_u32(uint32_t at, uint32_t v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

__device__ __forceinline__ uint64_t order_key(float v, int at) {
    return static_cast<uint64_t>(key_f32(__float_as_uint(v + 0.f))) << 32 | static_cast<uint32_t>(~at);  // -0 equals +0
}
__device__ __forceinline__ float key_value(uint64_t k) { return __uint_as_float(unkey_f32(static_cast<uint32_t>(k >> 32))); }
__device__ __forceinline__ int key_at(uint64_t k) { return static_cast<int>(~static_cast<uint32_t>(k)); }

// A word's numbers, none below -10 kFar: beside a larger one those have no part in the sums.
__device__ __forceinline__ void bounded(const uint4& q, float (&v)[4]) {
    unpack16(q, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = fmaxf(v[j], -10.f * kFar);
}
__device__ __forceinline__ void bounded(uint4 q, float (&v)[8]) {
    const __nv_bfloat162 least = __float2bfloat162_rn(-10.f * kFar);
    const auto raise = [&](uint32_t u) {
        const __nv_bfloat162 m = __hmax2(*reinterpret_cast<const __nv_bfloat162*>(&u), least);
        return *reinterpret_cast<const uint32_t*>(&m);
    };
    unpack16(make_uint4(raise(q.x), raise(q.y), raise(q.z), raise(q.w)), v);
}

// NT threads share a row's part.
template <int NT>
struct LogShared {
    uint4 hit[kLogHits];        // words with a number above the edge, and their numbers in the row
    int hit_word[kLogHits];
    uint64_t list[kLogList];
    uint64_t best[kLogMaxTop];  // the largest so far, in order
    float group[kLogGroups];
    uint64_t reduce[NT / 32];
    Part parts[NT / 32];
    uint32_t edge;              // as a key
    int count, kept, hits;
    // the row's first CTA: what every CTA of the cluster found, written by them
    Part all_parts[kLogCluster];
    int all_kept[kLogCluster];
    uint64_t all_best[kLogCluster * kLogMaxTop];
};

// The `top` largest of list[0 .. count), in order, to best[]: an entry's rank is the number of larger ones, which
// four threads count together.  Called by all threads; list and count are complete.  Returns what all
// later numbers have to exceed.
template <int NT>
__device__ __forceinline__ float cut_list(LogShared<NT>& sh, int count, int top) {
    const int part = threadIdx.x % 4;
    for (int i0 = 0; i0 < count; i0 += NT / 4) {
        const int i = i0 + static_cast<int>(threadIdx.x) / 4;
        const uint64_t k = i < count ? sh.list[i] : ~0ull;
        int above = 0;
#pragma unroll 4
        for (int j = part; j < count; j += 4) above += sh.list[j] > k ? 1 : 0;
        above += __shfl_xor_sync(kLanes, above, 1);
        above += __shfl_xor_sync(kLanes, above, 2);
        if (part == 0 && i < count && above < top) sh.best[above] = k;
    }
    const int kept = min(count, top);
    if (threadIdx.x == 0) sh.kept = kept;
    __syncthreads();
    return kept == top ? key_value(sh.best[top - 1]) : -INFINITY;
}

// A number that at least `top` of the CTA's present numbers reach, from the maxima of 64 groups of them (a
// thread's is `most`): the largest group maximum that `top` of them reach, -inf where there are too few.
template <int NT>
__device__ __forceinline__ float group_edge(LogShared<NT>& sh, float most, int top) {
    constexpr int GROUP = NT / kLogGroups;
    const int tid = threadIdx.x, lane = tid & 31;
    const float g = lanes_max<GROUP>(most);
    if (lane % GROUP == 0) sh.group[tid / GROUP] = g;
    if (tid == 0) sh.edge = 0u;
    __syncthreads();
    int reach = 0;  // how many maxima reach the thread's group's: the group's threads look at a part of them each
#pragma unroll
    for (int j = 0; j < kLogGroups / 4 / GROUP; ++j) {
        const float4 o = reinterpret_cast<const float4*>(sh.group)[(lane % GROUP) * (kLogGroups / 4 / GROUP) + j];
        reach += (o.x >= g ? 1 : 0) + (o.y >= g ? 1 : 0) + (o.z >= g ? 1 : 0) + (o.w >= g ? 1 : 0);
    }
#pragma unroll
    for (int d = 1; d < GROUP; d <<= 1) reach += __shfl_xor_sync(kLanes, reach, d);
    const uint32_t best = __reduce_max_sync(kLanes, reach >= top ? key_f32(__float_as_uint(g + 0.f)) : 0u);
    if (lane == 0) atomicMax(&sh.edge, best);
    __syncthreads();
    const uint32_t key = sh.edge;
    return key == 0u ? -INFINITY : __uint_as_float(unkey_f32(key));
}

// The `top` largest of best[0 .. kept) and of the listed words' numbers above `edge` (`equal`: at it too), to
// best[].  Returns the new edge; NaN where the list of words (or of numbers) was too short.
template <typename T, int NT>
__device__ __forceinline__ float cut_hits(LogShared<NT>& sh, float edge, bool equal, int shift, int top) {
    constexpr int PER = kPer<T>;
    const int tid = threadIdx.x;
    __syncthreads();
    const int hits = sh.hits, kept = sh.kept;
    if (hits > kLogHits) return NAN;
    if (hits + kept > kLogFew) {  // a higher edge, so that few numbers are left to rank
        float most = tid < kept ? key_value(sh.best[tid]) : -INFINITY;
        for (int h = tid; h < hits; h += NT) most = fmaxf(most, word_max<T>(sh.hit[h]));
        const float higher = group_edge(sh, most, top);
        if (higher > edge) edge = higher, equal = true;
    }
    if (tid == 0) sh.count = 0;
    __syncthreads();
    const auto put = [&](uint64_t k) {
        const int n = atomicAdd(&sh.count, 1);
        if (n < kLogList) sh.list[n] = k;
    };
    if (tid < kept && key_value(sh.best[tid]) >= edge) put(sh.best[tid]);
#pragma unroll 1
    for (int h = tid; h < hits; h += NT) {
        float v[PER];
        unpack16(sh.hit[h], v);
        const int at = sh.hit_word[h] * PER - shift;
#pragma unroll
        for (int j = 0; j < PER; ++j)
            if (equal ? v[j] >= edge : v[j] > edge) put(order_key(v[j], at + j));
    }
    __syncthreads();
    const int count = sh.count;
    if (tid == 0) sh.hits = 0;
    if (count > kLogList) return NAN;
    return cut_list(sh, count, top);
}

// The `top` largest of the CTAs' lists all_best[r * 32 ..], each in order: lane i of each warp gets the i-th, 0 for
// none.  Pairs of lists become one until one is left: an entry's rank is its own in its list and the number of
// larger ones in the other (binary search).
template <int NT>
__device__ __forceinline__ uint64_t merge_lists(LogShared<NT>& sh, int lists, int top) {
    static_assert(kLogList >= kLogCluster * kLogMaxTop / 2, "lists take turns in two arrays");
    const int lane = threadIdx.x & 31;
    uint64_t *from = sh.all_best, *to = sh.list;
    for (; lists > 1; lists /= 2) {
        for (int i = threadIdx.x; i < lists * kLogMaxTop; i += NT) {
            const int mine = i / kLogMaxTop, other = mine ^ 1, at = i % kLogMaxTop;
            const int kept = sh.all_kept[mine], others = sh.all_kept[other];
            if (at < kept) {
                const uint64_t k = from[i];
                int lo = 0, hi = others;  // the first of the other's entries below k
                while (lo < hi) {
                    const int mid = (lo + hi) / 2;
                    if (from[other * kLogMaxTop + mid] > k) lo = mid + 1;
                    else hi = mid;
                }
                if (at + lo < top) to[mine / 2 * kLogMaxTop + at + lo] = k;
            }
        }
        int kept = 0;
        if (threadIdx.x < lists / 2) kept = min(top, sh.all_kept[2 * threadIdx.x] + sh.all_kept[2 * threadIdx.x + 1]);
        __syncthreads();
        if (threadIdx.x < lists / 2) sh.all_kept[threadIdx.x] = kept;
        __syncthreads();
        uint64_t* const swap = from;
        from = to, to = swap;
    }
    return lane < sh.all_kept[0] ? from[lane] : 0;
}

// The `top` largest of words [first, last) of a row, to best[]: for rows where the list of words did not do
// (rising ones, or thousands of equal numbers).  Chunk by chunk: an edge from the chunk's maxima first;
// where even that leaves too many, one number at a time.
template <typename T, int NT>
__device__ __noinline__ void largest_slowly(LogShared<NT>& sh, const T* x, int first, int last, int shift, int V, int top) {
    constexpr int PER = kPer<T>, U = kLogHeld / PER;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    float edge = -INFINITY;
    int kept = 0;
    for (int g0 = first; g0 < last; g0 += NT * U) {
        __syncthreads();
        if (tid < kept) sh.list[tid] = sh.best[tid];
        if (tid == 0) sh.count = kept;
        float most = -INFINITY;
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
            const int g = g0 + u * NT + tid;
            if (g < last) most = fmaxf(most, word_max<T>(row_word(x, g, shift, V)));
        }
        // numbers at the edge of earlier chunks lose to those, at this chunk's they may win
        const float e = fmaxf(edge, group_edge(sh, most, top));
        const bool equal = e > edge;
        if (equal ? most >= e : most > e) {
#pragma unroll 1
            for (int u = 0; u < U; ++u) {
                const int g = g0 + u * NT + tid, at = g * PER - shift;
                float v[PER];
                unpack16(g < last ? row_word(x, g, shift, V) : no_word<T>(), v);
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (equal ? v[j] >= e : v[j] > e) {
                        const int n = atomicAdd(&sh.count, 1);
                        if (n < kLogList) sh.list[n] = order_key(v[j], at + j);
                    }
            }
        }
        __syncthreads();
        int count = sh.count;
        if (count > kLogList) {
            uint64_t below = ~0ull;
            count = kept;
            for (int i = 0; i < top; ++i) {
                uint64_t k = 0;
#pragma unroll 1
                for (int u = 0; u < U; ++u) {
                    const int g = g0 + u * NT + tid, at = g * PER - shift;
                    float v[PER];
                    unpack16(g < last ? row_word(x, g, shift, V) : no_word<T>(), v);
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
                for (int w = 0; w < NT / 32; ++w) k = sh.reduce[w] > k ? sh.reduce[w] : k;
                __syncthreads();
                if (k == 0) break;
                if (tid == 0) sh.list[count] = k;
                ++count;
                below = k;
            }
        }
        __syncthreads();
        edge = cut_list(sh, count, top);
        kept = min(count, top);
    }
}

template <typename T, int NT, bool TOP>
__global__ void __launch_bounds__(NT, 1024 / NT) ds_token_logprobs_kernel(const LogParams p) {
    constexpr int PER = kPer<T>, U = kLogHeld / PER, CHUNK = NT * U;
    __shared__ __align__(16) LogShared<NT> sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t ctas = gridDim.x, rank = blockIdx.x;  // of the row
    const int64_t row = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
    pdl_launch_dependents();
    if (row >= p.rows) return;  // a whole cluster
    if (TOP && tid == 0) sh.hits = sh.kept = 0;
    const T* x = static_cast<const T*>(p.x) + row * p.stride;
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(x) % 16 / sizeof(T));
    const int words = (p.V + shift + PER - 1) / PER;
    const int first = min(words, static_cast<int>(rank) * p.per_cta), last = min(words, first + p.per_cta);
    const int whole = min(last, (p.V + shift) / PER);  // words that end within the row
    if (ctas > 1) cluster_arrive();
    if (TOP) __syncthreads();
    pdl_wait();

    // the given token's logit: with the first words where a row's latency counts, else at the end
    float given = 0.f;
    int token = -1;
    const auto look_up = [&]() {
        token = p.tokens[row];
        if (token < 0 || token >= p.V) token = -1;
        else given = row_f32(x[token]);
    };
    if (tid == 0 && rank == 0 && ctas > 1) look_up();
    Part a = {-INFINITY, 0.f, 0.f};
    float edge = -INFINITY;  // at least `top` numbers seen reach it (or it is -inf): later ones have to exceed it
    bool reached = false;    // numbers at the edge itself are listed as well
    bool slow = false;       // the list was too short
    int chunk = 0, cut_at = 2;
    for (int g0 = first; g0 < last; g0 += CHUNK, ++chunk) {
        uint4 q[U];
        if (g0 > 0 && g0 + CHUNK <= whole) {
            const T* at = x + (static_cast<int64_t>(g0 + tid) * PER - shift);
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = *reinterpret_cast<const uint4*>(at + u * NT * PER);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int g = g0 + u * NT + tid;
                q[u] = g < last ? row_word(x, g, shift, p.V) : no_word<T>();
            }
        }
        float top_of[U], most = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) top_of[u] = word_max_or_nan<T>(q[u]), most = max_or_nan(most, top_of[u]);
        rise(a, most);
        if (most != most) {  // the row has no sums, and its top is found without the list of words
            a.s = NAN;
            if (TOP) atomicMax(&sh.hits, kLogHits + 1);
        } else if (!is_far(a.m)) {
            const Two nm = two(-a.m, -a.m), l2e = two(kLog2e, kLog2e);
            Two s = 0, w = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[PER];
                bounded(q[u], v);
#pragma unroll
                for (int j = 0; j < PER; j += 2) {
                    const Two y = mul_two(add_two(two(v[j], v[j + 1]), nm), l2e);
                    const Two e = two(exp2_term(lower(y)), exp2_term(upper(y)));
                    s = add_two(s, e);
                    w = fma_two(e, y, w);
                }
            }
            a.s += lower(s) + upper(s);
            a.w += lower(w) + upper(w);
        } else if (a.m > -INFINITY) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[PER];
                unpack16(q[u], v);
#pragma unroll
                for (int j = 0; j < PER; ++j) a.s += v[j] == a.m ? 1.f : 0.f;
            }
        }
        if (TOP && !slow) {
            if (chunk == 0) {
                edge = group_edge(sh, most, p.top);
                reached = edge > -INFINITY;
            }
            // words with a number above the edge are listed, of the first chunk those with one at it too
            const bool equal = chunk == 0 && reached;
            if (equal ? most >= edge : most > edge) {
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (equal ? top_of[u] >= edge : top_of[u] > edge) {
                        const int n = atomicAdd(&sh.hits, 1);
                        if (n < kLogHits) sh.hit[n] = q[u], sh.hit_word[n] = g0 + u * NT + tid;
                    }
            }
            // cut after 2, 8, 32 .. chunks and at the end: in between the list grows by a few times `top` where
            // numbers come in no order
            if (chunk + 1 == cut_at || g0 + CHUNK >= last) {
                if (chunk + 1 == cut_at) cut_at *= 4;
                edge = cut_hits<T>(sh, edge, reached, shift, p.top);
                reached = false;
                slow = edge != edge;
            }
        }
    }
    if constexpr (TOP) {
        if (slow) largest_slowly(sh, x, first, last, shift, p.V, p.top);
    }

    // the parts of a warp, of the CTA's warps, and of the cluster's CTAs: relative to their largest, then added
    const auto over = [](Part c, auto lanes) {
        constexpr int N = decltype(lanes)::value;
        rise(c, lanes_max<N>(c.m));
        return Part{c.m, lanes_sum<N>(c.s), lanes_sum<N>(c.w)};
    };
    const Part none = {-INFINITY, 0.f, 0.f};
    a = over(a, std::integral_constant<int, 32>());
    if (lane == 0) sh.parts[warp] = a;
    __syncthreads();
    Part all = none;
    if (warp == 0) all = over(lane < NT / 32 ? sh.parts[lane] : none, std::integral_constant<int, 32>());
    if (ctas > 1) {
        // to the row's first CTA
        cluster_wait();  // it runs
        if (tid == 0) {
            const uint32_t to = map_rank(&sh.all_parts[rank], 0);
            st_cluster_u32(to, __float_as_uint(all.m));
            st_cluster_u32(to + 4, __float_as_uint(all.s));
            st_cluster_u32(to + 8, __float_as_uint(all.w));
            if (TOP) st_cluster_u32(map_rank(&sh.all_kept[rank], 0), static_cast<uint32_t>(sh.kept));
        }
        if (TOP && tid < sh.kept) {
            const uint32_t to = map_rank(&sh.all_best[rank * kLogMaxTop + tid], 0);
            st_cluster_u32(to, static_cast<uint32_t>(sh.best[tid]));
            st_cluster_u32(to + 4, static_cast<uint32_t>(sh.best[tid] >> 32));
        }
        cluster_sync_all();
        if (rank != 0) return;
        if (warp == 0) all = over(lane < static_cast<int>(ctas) ? sh.all_parts[lane] : none, std::integral_constant<int, 32>());
        if constexpr (TOP) {
            const uint64_t mine = merge_lists(sh, static_cast<int>(ctas), p.top);
            if (warp == 0) {
                if (lane < p.top) sh.best[lane] = mine;
                if (lane == 0) sh.kept = sh.all_kept[0];
                __syncwarp();
            }
        }
    }
    if (warp != 0) return;
    if (all.m == INFINITY) all.s = NAN;  // inf - inf
    const bool some = all.s != 0.f, spoilt = all.s != all.s;
    const float logs = some ? log2f(all.s) : 0.f;
    const auto log_p = [&](float v) { return some ? (v - all.m) - logs * kLn2 : -INFINITY; };
    if (tid == 0) {
        if (ctas == 1) look_up();
        p.logprobs[row] = token >= 0 ? log_p(given) : 0.f;
        p.lse[row] = all.m + logs * kLn2;
        const float H = (logs - all.w / all.s) * kLn2;
        p.entropy[row] = spoilt ? NAN : some && H > 0.f ? H : 0.f;
    }
    if constexpr (TOP) {
        int at = 0, have = 0;  // the lane's token, and how many lanes have theirs
        if (spoilt) {  // the NaN ones come first
            for (int i0 = 0; have < p.top && i0 < p.V; i0 += 32 * 8) {
                float v[8];
                bool any = false;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    v[u] = i0 + u * 32 + lane < p.V ? row_f32(x[i0 + u * 32 + lane]) : 0.f;
                    any |= v[u] != v[u];
                }
                if (!__any_sync(kLanes, any)) continue;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const uint32_t which = __ballot_sync(kLanes, v[u] != v[u]);
                    const int n = __popc(which);
                    if (lane >= have && lane < have + n) at = i0 + u * 32 + static_cast<int>(__fns(which, 0, lane - have + 1));
                    have += n;
                }
            }
        }
        const int numbers = lane - have;  // its place among the numbers
        const bool real = numbers >= 0 && lane < p.top && numbers < sh.kept;
        const uint64_t k = real ? sh.best[numbers] : 0;
        const float v = real ? key_value(k) : -INFINITY;
        if (real) at = key_at(k);
        // fewer numbers above -inf than asked for: the first of the others follow
        have += __popc(__ballot_sync(kLanes, real));
        for (int i0 = 0; have < p.top && i0 < p.V; i0 += 32) {
            const bool other = i0 + lane < p.V && row_f32(x[i0 + lane]) == -INFINITY;
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
// One number in, one out; a CTA takes a run of one row.  log p = x - lse, and lse is rounded to fp32: up to
// |lse| = 64 that moves every p of the row by at most 2^-19 of itself.  A row beyond (logits with a common
// offset, a row masked with -1e9 throughout: lse = m, and what it lost is log V) has one CTA, which first
// sums exp(x - lse) over it: log p = (x - lse) - log of that sum.  Memory bounds both: 2048 x 129280 bf16 in 153 us,
// in 286 where every row is summed again (a row alone, by one CTA: 30 us, 2.7 without).
constexpr int kBackThreads = 256, kBackWords = 4;
constexpr float kLseKept = 64.f;

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

// A row with what its gradient takes.
template <typename T>
struct BackRow {
    const T* x;
    T* out;
    int V, t;      // t: the given token, -1 for none
    float g, h, H, lse;
    float rest;    // log sum exp(x - lse), where lse is not enough
    bool none;     // a row of -inf alone has no probabilities: no gradient
    int shift;     // numbers before the row's start in its first 16 bytes
};

// A thread's words of run number `run` of a row.
template <typename T>
__device__ __forceinline__ void load_run(const BackRow<T>& r, int run, uint4 (&q)[kBackWords]) {
    const int words = (r.V + r.shift + kPer<T> - 1) / kPer<T>, w0 = run * (kBackThreads * kBackWords);
#pragma unroll
    for (int u = 0; u < kBackWords; ++u) {
        const int w = w0 + u * kBackThreads + threadIdx.x;
        q[u] = w < words ? row_word(r.x, w, r.shift, r.V) : no_word<T>();
    }
}

// The gradient of the run whose words are q (VEC; else they are not used); REST: with the row's rest.
template <typename T, bool VEC, bool REST>
__device__ __forceinline__ void put_run(const BackRow<T>& r, int run, const uint4 (&q)[kBackWords]) {
    constexpr int PER = kPer<T>, U = kBackWords;
    // -p (g + h (log p + H)), with log p bounded so that 0 times it stays 0; NaN where lse is
    const auto grad_of = [&](float v) {
        const float lp = max_or_nan(REST ? (v - r.lse) - r.rest : v - r.lse, -150.f);
        return -exp2_term(lp * kLog2e) * fmaf(r.h, lp + r.H, r.g);
    };
    if (VEC) {
        // both rows lie alike against 16-byte boundaries
        const int words = (r.V + r.shift + PER - 1) / PER, w0 = run * (kBackThreads * U);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int w = w0 + u * kBackThreads + threadIdx.x, at = w * PER - r.shift;
            if (w >= words) break;
            float v[PER];
            unpack16(q[u], v);
#pragma unroll
            for (int j = 0; j < PER; ++j) v[j] = r.none ? 0.f : grad_of(v[j]);
            if (!r.none && r.t >= at && r.t < at + PER) {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (at + j == r.t) v[j] += r.g;
            }
            if (at >= 0 && at + PER <= r.V) {
                *reinterpret_cast<uint4*>(r.out + at) = pack16(v);
            } else {
#pragma unroll
                for (int j = 0; j < PER; ++j)
                    if (at + j >= 0 && at + j < r.V) row_put(r.out + at + j, v[j]);
            }
        }
    } else {
        const int64_t c0 = static_cast<int64_t>(run) * (kBackThreads * U * PER);
#pragma unroll 8
        for (int i = 0; i < U * PER; ++i) {
            const int64_t c = c0 + i * kBackThreads + threadIdx.x;
            if (c < r.V) row_put(r.out + c, r.none ? 0.f : grad_of(row_f32(r.x[c])) + (c == r.t ? r.g : 0.f));
        }
    }
}

// A row whose lse is not enough, by one CTA.
template <typename T, bool VEC>
__device__ __noinline__ void put_row(BackRow<T> r, int runs) {
    __shared__ float sh_sum[kBackThreads / 32];
    uint4 q[kBackWords];
    float sum = 0.f;
    for (int run = 0; run < runs; ++run) {
        load_run(r, run, q);
#pragma unroll
        for (int u = 0; u < kBackWords; ++u) {
            float v[kPer<T>];
            unpack16(q[u], v);
#pragma unroll
            for (int j = 0; j < kPer<T>; ++j) sum += exp2_term((v[j] - r.lse) * kLog2e);
        }
    }
    sum = lanes_sum<32>(sum);
    if (threadIdx.x % 32 == 0) sh_sum[threadIdx.x / 32] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < kBackThreads / 32; ++w) sum += sh_sum[w];
    r.rest = log2f(sum) * kLn2;
    for (int run = 0; run < runs; ++run) {
        if (VEC) load_run(r, run, q);
        put_run<T, VEC, true>(r, run, q);
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(kBackThreads) ds_token_logprobs_backward_kernel(const LogBackParams p) {
    pdl_launch_dependents();
    pdl_wait();
    const int64_t row = blockIdx.x / p.runs;
    const int run = static_cast<int>(blockIdx.x % p.runs);
    BackRow<T> r;
    r.x = static_cast<const T*>(p.x) + row * p.stride;
    r.out = static_cast<T*>(p.out) + row * p.out_stride;
    r.V = p.V;
    r.shift = static_cast<int>(reinterpret_cast<uintptr_t>(r.x) % 16 / sizeof(T));
    const float lse = p.lse[row];
    uint4 q[kBackWords];
    if (VEC) load_run(r, run, q);  // on their way while lse is looked at (2048 x 129280 bf16: 158 us else, 153)
    r.t = p.tokens[row];
    r.g = p.grad[row], r.h = 0.f, r.H = 0.f;
    if (p.grad_entropy) r.h = p.grad_entropy[row], r.H = p.entropy[row];
    if (r.t < 0 || r.t >= p.V) r.t = -1, r.g = 0.f;
    r.none = lse == -INFINITY;
    r.lse = r.none ? 0.f : lse;
    r.rest = 0.f;
    const float size = fabsf(r.lse);
    if (size > kLseKept && size < INFINITY) {
        if (run == 0) put_row<T, VEC>(r, p.runs);
        return;
    }
    put_run<T, VEC, false>(r, run, q);
}

// ---------------------------------------------------------------- host --------------
template <typename T>
static ds_status launch_logprobs(LogParams p, int sms, cudaStream_t stream) {
    // rows that are many have a CTA of kLogFewThreads each: they take turns on an SM, and their barriers are between
    // fewer warps; else a cluster to a row, as many larger CTAs as give every SM two, of 32 numbers a thread at
    // least (4099 x 32003 bf16 with one token: 64 us with 128 threads, 73 with 256; one row of 129280 fp32 with 20:
    // 11.5 and 7.7)
    constexpr int PER = kPer<T>, CHUNK = kLogThreads * kLogHeld;
    const int64_t words = (static_cast<int64_t>(p.V) + 2 * PER - 2) / PER;
    int ctas = 1;
    while (ctas < kLogCluster && p.rows * ctas < 2 * sms && static_cast<int64_t>(ctas) * CHUNK < p.V) ctas *= 2;
    p.per_cta = static_cast<int32_t>((words + ctas - 1) / ctas);
    const unsigned y = static_cast<unsigned>(p.rows < 65535 ? p.rows : 65535);
    const dim3 grid(ctas, y, static_cast<unsigned>((p.rows + y - 1) / y));
    if (ctas == 1 && p.rows >= 2 * sms) {
        const auto kern = p.top > 0 ? ds_token_logprobs_kernel<T, kLogFewThreads, true> : ds_token_logprobs_kernel<T, kLogFewThreads, false>;
        return launch_pdl(kern, grid, kLogFewThreads, 0, 1, stream, p);
    }
    const auto kern = p.top > 0 ? ds_token_logprobs_kernel<T, kLogThreads, true> : ds_token_logprobs_kernel<T, kLogThreads, false>;
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
    const int64_t per = 16 / es, words = (V + 2 * per - 2) / per, runs = (words + kBackThreads * kBackWords - 1) / (kBackThreads * kBackWords);
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
