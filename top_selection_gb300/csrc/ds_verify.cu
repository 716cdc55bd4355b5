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
// A cluster of C CTAs takes a sequence, each CTA a slice of the vocabulary.  Rows go in rounds of
// R: each CTA finds its slice's maximum and sum of exponentials of the round's rows in one pass
// (online: a thread rescales its sum when its maximum rises), the cluster exchanges these over
// distributed shared memory, and every CTA decides by itself where the sequence stops, by the same
// arithmetic in the same order.  Rows behind the stop's round, which the answer does not need, are
// not read.  The stop row is read a second time for the race, from L2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <atomic>
#include <type_traits>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerRound = 8;                  // most rows of a round
constexpr int kVerCluster = 16;               // most CTAs of a sequence
constexpr uint32_t kWarp = 0xFFFFFFFFu;

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
    int32_t C, R;                    // CTAs of a sequence, rows of a round
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

__device__ __forceinline__ float ver_exp2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// (x + add) * by and a + b, two numbers to an instruction
__device__ __forceinline__ float2 scaled2(float x, float y, float add, float by) {
    float2 r;
    asm("{\n\t.reg .b64 x, a, b;\n\t"
        "mov.b64 x, {%2, %3};\n\tmov.b64 a, {%4, %4};\n\tmov.b64 b, {%5, %5};\n\t"
        "add.rn.f32x2 x, x, a;\n\tmul.rn.f32x2 x, x, b;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x), "f"(y), "f"(add), "f"(by));
    return r;
}
__device__ __forceinline__ float2 sum2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float ver_max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A row's (or a slice's) largest logit, its first place (temperature 0 only), and the sum of
// exp((x - m) / temperature); m = -inf and s = 0 where every logit is -inf.
struct RowStat {
    float m, s;
    int at;
};

// The statistics of two disjoint slices as one; c = log2(e) / temperature.
__device__ __forceinline__ RowStat both_stats(RowStat a, RowStat b, float c) {
    RowStat r;
    r.m = fmaxf(a.m, b.m);
    r.at = a.m > b.m ? a.at : b.m > a.m ? b.at : min(a.at, b.at);
    r.s = (a.m > -INFINITY ? a.s * ver_exp2((a.m - r.m) * c) : 0.f) +
          (b.m > -INFINITY ? b.s * ver_exp2((b.m - r.m) * c) : 0.f);
    return r;
}
// The lanes' statistics as one, in every lane.  The maximum goes by its order-preserving key.
__device__ __forceinline__ RowStat warp_stats(RowStat a, float c, bool greedy) {
    const float m = __uint_as_float(unkey_f32(__reduce_max_sync(kWarp, key_f32(__float_as_uint(a.m)))));
    if (greedy) return {m, 0.f, static_cast<int>(__reduce_min_sync(kWarp, a.m == m ? static_cast<uint32_t>(a.at) : 0x7FFFFFFFu))};
    float s = a.m > -INFINITY ? a.s * ver_exp2((a.m - m) * c) : 0.f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(kWarp, s, d);
    return {m, s, 0x7FFFFFFF};
}

// The numbers of a 16-byte word as fp32.
template <typename T>
struct Vec {
    static constexpr int N = 16 / sizeof(T);
    static __device__ __forceinline__ void unpack(uint4 w, float* x) {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(u[i]);
            } else {
                x[2 * i] = __uint_as_float(u[i] << 16);
                x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
            }
        }
    }
};

// Adds M words of N numbers to a thread's statistics; word k's first place is first + k * step.
template <int M, int N, bool GREEDY>
__device__ __forceinline__ void add_numbers(RowStat& a, const float (&x)[M][N], int first, int step, float c) {
    float top = x[0][0];
#pragma unroll
    for (int k = 0; k < M; ++k)
#pragma unroll
        for (int i = k == 0; i < N; i += 2) top = i + 1 < N ? ver_max3(top, x[k][i], x[k][i + 1]) : fmaxf(top, x[k][i]);
    if (GREEDY) {
        if (top > a.m) {  // a thread's places ascend: a later equal number is not the first
            a.m = top;
#pragma unroll
            for (int k = M - 1; k >= 0; --k)
#pragma unroll
                for (int i = N - 1; i >= 0; --i)
                    if (x[k][i] == top) a.at = first + k * step + i;
        }
        return;
    }
    if (top > a.m) {
        a.s *= ver_exp2((a.m - top) * c);
        a.m = top;
    }
    if (a.m > -INFINITY) {
        if constexpr (N == 1) {
            a.s += ver_exp2((x[0][0] - a.m) * c);
        } else {
            float2 sum = make_float2(a.s, 0.f);
#pragma unroll
            for (int k = 0; k < M; ++k)
#pragma unroll
                for (int i = 0; i < N; i += 2) {
                    const float2 y = scaled2(x[k][i], x[k][i + 1], -a.m, c);
                    sum = sum2(sum, make_float2(ver_exp2(y.x), ver_exp2(y.y)));
                }
            a.s = sum.x + sum.y;
        }
    }
}

// CTA `part`'s slice of a row of V numbers: 16-byte words from the first aligned place on; the
// numbers before and behind the words fall to the first CTA.
template <typename T>
struct Slice {
    static constexpr int N = Vec<T>::N;
    const T* x;
    int V, head, words, from, to;
    __device__ __forceinline__ Slice(const T* x, int V, int part, int parts) : x(x), V(V) {
        const uint32_t past = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(x)) & 15u;
        head = min(V, static_cast<int>((16u - past) & 15u) / static_cast<int>(sizeof(T)));
        words = (V - head) / N;
        from = static_cast<int>(static_cast<int64_t>(words) * part / parts);
        to = static_cast<int>(static_cast<int64_t>(words) * (part + 1) / parts);
    }
    // U words from `at` on, one a thread; -inf behind the slice
    template <int U>
    __device__ __forceinline__ void load(int at, uint4 (&q)[U]) const {
        constexpr uint32_t none = sizeof(T) == 4 ? 0xFF800000u : 0xFF80FF80u;
        const uint4* w = reinterpret_cast<const uint4*>(x + head);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            q[u] = make_uint4(none, none, none, none);
            if (at + u * kVerThreads < to) q[u] = w[at + u * kVerThreads];
        }
    }
    // the number outside the words that is this thread's, if it has one
    __device__ __forceinline__ int outside() const {
        const int tid = threadIdx.x, place = tid < head ? tid : head + words * N + tid - head;
        return place < V ? place : -1;
    }
};

// Each warp's statistics of the CTA's slices of `rows` rows, into `out`.  A thread loads the next
// words, of the same row or the next, while it works on the last.
template <typename T, bool GREEDY>
__device__ __forceinline__ void rows_stats(const T* x0, int64_t stride, int rows, int V, int part, int parts, float c,
                                           RowStat (*out)[kVerWarps]) {
    constexpr int N = Vec<T>::N, U = 4, W = 16 / N, STEP = U * kVerThreads;  // W words at a time
    const int tid = threadIdx.x;
    Slice<T> next(x0, V, part, parts);
    int at = next.from + tid;
    uint4 q[U];
    next.load(at, q);
    for (int i = 0; i < rows; ++i) {
        const Slice<T> s = next;
        RowStat a = {-INFINITY, 0.f, 0x7FFFFFFF};
        // every thread takes the same steps (what lies behind the slice is -inf)
        for (int base = s.from; base < s.to || base == s.from; base += STEP) {
            uint4 now[U];
#pragma unroll
            for (int u = 0; u < U; ++u) now[u] = q[u];
            const int here = base + tid;
            if (base + STEP < s.to) {
                s.load(here + STEP, q);
            } else if (i + 1 < rows) {
                next = Slice<T>(x0 + (i + 1) * stride, V, part, parts);
                next.load(next.from + tid, q);
            }
#pragma unroll
            for (int u = 0; u < U; u += W) {
                float y[W][N];
#pragma unroll
                for (int k = 0; k < W; ++k) Vec<T>::unpack(now[u + k], y[k]);
                add_numbers<W, N, GREEDY>(a, y, s.head + (here + u * kVerThreads) * N, kVerThreads * N, c);
            }
        }
        if (part == 0) {
            const int place = s.outside();
            if (place >= 0) {
                const float one[1][1] = {{ver_f32(s.x[place])}};
                RowStat b = {-INFINITY, 0.f, 0x7FFFFFFF};
                add_numbers<1, 1, GREEDY>(b, one, place, 0, c);
                a = both_stats(a, b, c);
            }
        }
        a = warp_stats(a, c, GREEDY);
        if ((tid & 31) == 0) out[i][tid >> 5] = a;
    }
}

struct Race {
    float v;
    int i;
};
__device__ __forceinline__ Race warp_best(Race a) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        best_of(a.v, a.i, __shfl_xor_sync(kWarp, a.v, d), __shfl_xor_sync(kWarp, a.i, d));
    return a;
}

// Four numbers from place v on, in one load where `vec`.
__device__ __forceinline__ void four(const float* p, bool vec, float (&x)[4]) {
    if (vec) {
        const float4 w = *reinterpret_cast<const float4*>(p);
        x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = p[i];
    }
}
__device__ __forceinline__ void four(const __nv_bfloat16* p, bool vec, float (&x)[4]) {
    if (vec) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        x[0] = __uint_as_float(w.x << 16), x[1] = __uint_as_float(w.x & 0xFFFF0000u);
        x[2] = __uint_as_float(w.y << 16), x[3] = __uint_as_float(w.y & 0xFFFF0000u);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = ver_f32(p[i]);
    }
}

// A thread's best of r / e over CTA `part`'s slice; q null: the draft is one-hot at t (t < 0: r = p).
// Places go in groups of four from the first one where the noise is aligned to 16 bytes; the logits
// and q, whose rows may lie otherwise, are read four at a time where both are aligned there too.
template <typename T>
__device__ __forceinline__ Race slice_race(const T* x, const float* q, int t, const float* e, int V, int part, int parts,
                                           float m, float c, float inv_s) {
    float br = 0.f, be = 1.f;  // the best so far
    int bi = 0x7FFFFFFF;
    // r / e against br / be by cross products: no quotient, no branch (a thread's bests change
    // often while it has seen few places, and some lane's always does)
    const auto one = [&](int v, float xv, float qv, float ev) {
        const float r = fmaf(ver_exp2((xv - m) * c), inv_s, -qv);
        const bool wins = r * be > br * ev;
        br = wins ? r : br;
        be = wins ? ev : be;
        bi = wins ? v : bi;
    };
    const int head = min(V, static_cast<int>((16u - (reinterpret_cast<uintptr_t>(e) & 15u)) & 15u) / 4);
    const int groups = (V - head) / 4;
    const int from = static_cast<int>(static_cast<int64_t>(groups) * part / parts);
    const int to = static_cast<int>(static_cast<int64_t>(groups) * (part + 1) / parts);
    const T* xg = x + head;
    const float *eg = e + head, *qg = q ? q + head : nullptr;
    const bool vec = (reinterpret_cast<uintptr_t>(xg) & (4 * sizeof(T) - 1)) == 0 &&
                     (reinterpret_cast<uintptr_t>(qg) & 15u) == 0;
    const auto groups_at = [&](int g, auto count, auto wide) {  // loads of `count` groups in flight
        constexpr int M = decltype(count)::value;
        float xv[M][4], qv[M][4], ev[M][4];
#pragma unroll
        for (int k = 0; k < M; ++k) {
            const int at = (g + k * kVerThreads) * 4;
            four(xg + at, wide.value, xv[k]);
            four(eg + at, true, ev[k]);
            if (q) four(qg + at, wide.value, qv[k]);
        }
#pragma unroll
        for (int k = 0; k < M; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int v = head + (g + k * kVerThreads) * 4 + i;
                one(v, xv[k][i], q ? qv[k][i] : v == t ? 1.f : 0.f, ev[k][i]);
            }
    };
    int g = from + static_cast<int>(threadIdx.x);
    const auto all = [&](auto wide) {
        for (; g + kVerThreads < to; g += 2 * kVerThreads) groups_at(g, std::integral_constant<int, 2>{}, wide);
        for (; g < to; g += kVerThreads) groups_at(g, std::integral_constant<int, 1>{}, wide);
    };
    if (vec) all(std::true_type{});
    else all(std::false_type{});
    Race a = {br / be, bi};
    const int tid = threadIdx.x, v = tid < head ? tid : head + groups * 4 + tid - head;
    if (part == 0 && v < V) {  // a thread's places do not ascend here
        br = 0.f, be = 1.f, bi = 0x7FFFFFFF;
        one(v, ver_f32(x[v]), q ? q[v] : v == t ? 1.f : 0.f, e[v]);
        best_of(a.v, a.i, br / be, bi);
    }
    return a;
}

template <typename T>
__global__ void __launch_bounds__(kVerThreads, 2) ds_verify_kernel(const VerifyParams p) {
    __shared__ RowStat sh_warp[kVerRound][kVerWarps];  // each warp's statistics of the round's rows
    __shared__ RowStat sh_cta[2][kVerRound];           // the CTA's, for the cluster; by the round's parity
    __shared__ RowStat sh_stop;                        // the stop row's
    __shared__ Race sh_race[kVerWarps];
    __shared__ Race sh_best[2];                        // the CTA's, for the cluster; by the attempt
    __shared__ int sh_n;                               // accepted rows of the round
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t b = blockIdx.x / static_cast<uint32_t>(p.C);
    const int part = static_cast<int>(blockIdx.x - b * p.C);
    const auto sync_all = [&]() {
        if (p.C > 1) cluster_sync_all();
        else __syncthreads();
    };
    pdl_launch_dependents();
    pdl_wait();
    const float temp = p.temps ? p.temps[b] : p.temperature;
    const bool greedy = !(temp > 0.f);
    // a temperature too small for its inverse separates any two logits all the same
    const float inv_t = greedy ? 1.f : fminf(1.f / temp, 1e30f);
    const float c = inv_t * 1.4426950408889634f;
    const int len = p.lens ? min(max(p.lens[b], 0), p.S) : p.S;
    const T* seq = static_cast<const T*>(p.logits) + b * p.seq_stride;
    int32_t* tokens = p.tokens + b * (p.S + 1);
    float* probs = p.probs ? p.probs + b * (p.S + 1) : nullptr;

    int n = 0;
    for (int round = 0;; ++round) {
        const int rows = min(p.R, len + 1 - n);
        // warp 0, lane i: the round's i-th draft, fetched while the rows are read
        int t = -1;
        float u = 0.f, qt = 1.f, xt = -INFINITY;
        if (warp == 0 && lane < rows && n + lane < len) {
            t = p.drafts[b * p.S + n + lane];
            u = p.uniforms[b * p.S + n + lane];
            if (t < 0 || t >= p.V) t = -1;  // no column: refused
            if (t >= 0) {
                xt = ver_f32(seq[(n + lane) * p.row_stride + t]);
                if (p.q) qt = p.q[b * p.q_seq + (n + lane) * p.q_row + t];
            }
        }
        const T* x0 = seq + n * p.row_stride;
        if (greedy) rows_stats<T, true>(x0, p.row_stride, rows, p.V, part, p.C, c, sh_warp);
        else rows_stats<T, false>(x0, p.row_stride, rows, p.V, part, p.C, c, sh_warp);
        __syncthreads();
        RowStat* mine = sh_cta[round & 1];
        if (warp < rows) {
            RowStat a = {-INFINITY, 0.f, 0x7FFFFFFF};
            if (lane < kVerWarps) a = sh_warp[warp][lane];
            a = warp_stats(a, c, greedy);
            if (lane == 0) mine[warp] = a;
        }
        sync_all();
        if (warp == 0) {
            RowStat a = {-INFINITY, 0.f, 0x7FFFFFFF};
            if (lane < rows) {
                a = mine[lane];
                if (p.C > 1) {
                    a = {-INFINITY, 0.f, 0x7FFFFFFF};
                    for (int k = 0; k < p.C; ++k) {  // in one order in every CTA: the same decision
                        const uint32_t at = map_rank(&mine[lane], k);
                        a = both_stats(a, {__uint_as_float(ld_cluster_u32(at)), __uint_as_float(ld_cluster_u32(at + 4)),
                                           static_cast<int>(ld_cluster_u32(at + 8))}, c);
                    }
                }
            }
            float pt = 0.f;
            if (t >= 0 && a.m > -INFINITY) pt = greedy ? (t == a.at ? 1.f : 0.f) : expf((xt - a.m) * inv_t) / a.s;
            const bool ok = lane < rows && n + lane < len && u * qt < pt;
            const int run = __ffs(~__ballot_sync(kWarp, ok)) - 1;  // accepted rows in front (at most 8)
            if (part == 0 && lane < run) {
                tokens[n + lane] = t;
                if (probs) probs[n + lane] = pt;
            }
            if (lane == min(run, rows - 1)) sh_stop = a;
            if (lane == 0) sh_n = run;
        }
        __syncthreads();
        const int run = sh_n;
        n += run;
        if (run < rows) break;
    }

    // the stop row
    const RowStat stop = sh_stop;
    const T* x = seq + n * p.row_stride;
    int last = -1;
    if (greedy) {
        last = stop.m > -INFINITY ? stop.at : -1;
    } else if (stop.m > -INFINITY) {
        const bool refused = n < len;
        const float* e = p.noise + b * p.noise_stride;
        const float* q = refused && p.q ? p.q + b * p.q_seq + n * p.q_row : nullptr;
        int t = refused && !p.q ? p.drafts[b * p.S + n] : -1;
        const float inv_s = 1.f / stop.s;
        for (int attempt = 0; attempt < 2; ++attempt) {  // the second: r was 0 everywhere, so p itself
            Race a = slice_race(x, q, t, e, p.V, part, p.C, stop.m, c, inv_s);
            a = warp_best(a);
            if (lane == 0) sh_race[warp] = a;
            __syncthreads();
            if (warp == 0) {
                a = {0.f, 0x7FFFFFFF};
                if (lane < kVerWarps) a = sh_race[lane];
                a = warp_best(a);
                if (lane == 0) sh_best[attempt] = a;
            }
            sync_all();
            a = sh_best[attempt];
            for (int k = 0; k < p.C && p.C > 1; ++k) {
                const uint32_t at = map_rank(&sh_best[attempt], k);
                best_of(a.v, a.i, __uint_as_float(ld_cluster_u32(at)), static_cast<int>(ld_cluster_u32(at + 4)));
            }
            if (a.i < p.V) {
                last = a.i;
                break;
            }
            q = nullptr;
            t = -1;
        }
    }
    if (part == 0 && warp == 0) {
        float pl = 0.f;
        if (last >= 0) pl = greedy ? 1.f : expf((ver_f32(x[last]) - stop.m) * inv_t) / stop.s;
        for (int i = n + lane; i <= p.S; i += 32) {
            tokens[i] = i == n ? last : -1;
            if (probs) probs[i] = i == n ? pl : 0.f;
        }
        if (lane == 0) p.accepted[b] = n;
    }
    if (p.C > 1) cluster_sync_all();  // no CTA leaves while another may read its shared memory
}

template <typename T>
static ds_status launch_verify(const VerifyParams& p, int dev, int64_t sequences, cudaStream_t stream) {
    // clusters above 8 are a kernel's opt-in on a device: set once
    static std::atomic<bool> opted[64];
    if (p.C > 8 && !opted[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(ds_verify_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
            return DS_ERR_CUDA;
        opted[dev].store(true, std::memory_order_release);
    }
    return launch_pdl(ds_verify_kernel<T>, dim3(static_cast<unsigned>(sequences * p.C)), kVerThreads, 0, p.C, stream, p);
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
    int dev = 0;
    DevInfo info;
    if (cudaGetDevice(&dev) != cudaSuccess || !dev_info(dev, info)) return DS_ERR_CUDA;
    VerifyParams p = {};
    p.logits = logits;
    p.seq_stride = seq_stride;
    p.row_stride = row_stride;
    p.q = draft_probs;
    p.q_seq = probs_seq_stride;
    p.q_row = probs_row_stride;
    p.drafts = drafts;
    p.lens = draft_lens;
    p.uniforms = uniforms;
    p.noise = noise;
    p.noise_stride = noise_stride;
    p.temps = temperatures;
    p.temperature = temperature;
    p.S = S;
    p.V = static_cast<int32_t>(V);
    p.tokens = out_tokens;
    p.accepted = out_accepted;
    p.probs = out_probs;
    // CTAs of a sequence: as many as fit the GPU at once (two to an SM) with slices of at least 2048
    // numbers.  64 sequences of 129280 logits: 1 CTA each 78.7 us, 2 51.0, 4 37.4, 8 (two waves) 48.1.
    p.C = 1;
    while (p.C < kVerCluster && sequences * p.C * 2 <= 2 * info.sms && V / (p.C * 2) >= 2048) p.C *= 2;
    // rows of a round: all where CTAs are few and latency counts (one sequence of 4 drafts, 16 CTAs:
    // 13.4 us, with one row to a round 21.3); else two, one of which may be read in vain, for one
    // exchange less (64 sequences: 37.1 us, one 39.0, all 38.0; 200 of 5 short drafts 25.2, 26.0, 33.0)
    p.R = sequences * p.C <= info.sms ? kVerRound : 2;
    if (sequences * p.C > 0x7FFFFFFFLL) return DS_ERR_UNSUPPORTED;
    return dtype == DS_BF16 ? launch_verify<__nv_bfloat16>(p, dev, sequences, stream)
                            : launch_verify<float>(p, dev, sequences, stream);
}

}  // extern "C"
