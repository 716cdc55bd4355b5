// ds_attend.cu -- attention of new tokens over a paged cache of 4-bit keys and values
// (ds_cache_attention): every position of the context, or the positions a top-k selected.
//
// A key row of the cache stands for s c + m (codes c, bf16 scale s and minimum m, see
// ds_cache.cu), so a query row q scores it as
//     q . (s c + m) = s (q . (c - 8)) + (m + 8 s) (sum q),
// and a value row with weight p adds
//     p (s c + m) = (p s) (c - 8) + p (m + 8 s).
// The products are small whole numbers, exact in bf16, against q and against p s; the minima
// enter through one scalar per row (sum q, and the running sum of p (m + 8 s)).  The codes
// never leave registers: with tokens as the rows of the matrix instruction, the four lanes
// that share a fragment row read a token's codes as they lie in memory (any order of the
// contracted dimension serves, as long as q is read in the same order), and a masked OR turns
// two codes into two bf16 numbers 128 + c.
//
// m16n8k16 (mma.sync) rather than tcgen05: a step has 8 to 32 query rows per key head, the
// operand that streams is the cache, and tcgen05 takes it from shared memory only, so each
// tile would be expanded to four times its bytes, stored and read back.  Here a byte of the
// cache is loaded once into the register it is used from.
//
// Rows: the query rows that share a key head (heads of a group, and for whole contexts the
// tokens of the step as well) in tiles of 8; a CTA takes up to 8 * NT of them and one split of
// the positions; its warps take tiles of 32 positions in turn.  Softmax runs online per warp:
// one running maximum per row, raised only when a score passes it by 2^8 (the weights stay
// below 2^8 then, far from fp32's and bf16's ends), sums per lane.  Warps are joined in shared
// memory, splits by a second kernel.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kAttWarps = 4;
constexpr int kAttTile = 32;                   // positions per warp and step
constexpr uint32_t kNoEntry = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.0f;                 // in powers of two

struct AttendParams {
    const void* q;
    int64_t q_seq, q_tok, q_head;  // element strides
    const uint8_t* cache;
    const uint32_t* scales;        // two words per entry: key (s, m), value (s, m)
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lens;
    const int32_t* indices;        // [B, Q, K] or null
    void* out;
    float* lse;
    float* ws_o;                   // split partials: [unit][split][rows][D]
    float* ws_ml;                  //                 [unit][split][rows][2]
    int64_t max_pos;               // table width * page
    int32_t Q, K, heads, group, page_log, pages;
    int32_t rows;                  // query rows per unit before tiling
    int32_t row_groups, splits, chunk;
    float scale;
};

__device__ __forceinline__ float att_f32(float v) { return v; }
__device__ __forceinline__ float att_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Codes at bit 4 * i of both halves of w -> two bf16 numbers c - 8.
__device__ __forceinline__ uint32_t codes_bf16(uint32_t w, int i) {
    const uint32_t x = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;  // 128 + c
    const __nv_bfloat162 a = *reinterpret_cast<const __nv_bfloat162*>(&x);
    const __nv_bfloat162 r = __hsub2(a, __floats2bfloat162_rn(136.f, 136.f));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// 2^x with a relative error of 2^-22: an error the weight has already from its argument.
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// x = the sum of NS bf16 parts (8 bits of x each), two numbers at a time
template <int NS>
__device__ __forceinline__ void split_bf16(float a, float b, uint32_t (&part)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        part[i] = pack_bf16(a, b);
        if (i + 1 < NS) {
            a -= __uint_as_float(part[i] << 16);
            b -= __uint_as_float(part[i] & 0xFFFF0000u);
        }
    }
}

template <int D>
struct AttTile {
    uint32_t k[4][D / 32];  // tokens g + 8 i, the lane's quarter of the key row
    uint32_t v[8][D / 64];  // tokens 16 j + {2t, 2t+1, 2t+8, 2t+9}, the lane's eighth of the value row
    uint2 sc;               // token `lane`: key and value (s, m)
    int pos;                // token `lane`: its position, or INT_MAX
};

template <int D>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[D]) {
    if constexpr (D % 4 == 0) {
#pragma unroll
        for (int i = 0; i < D / 4; ++i) {
            const uint4 q = reinterpret_cast<const uint4*>(p)[i];
            w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
        }
    } else if constexpr (D == 2) {
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[0] = q.x, w[1] = q.y;
    } else {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
}

// T: type of q and out.  NQ / NP: bf16 parts of q and of the weights (q in bf16: 1 part is
// exact; weights in two parts keep 16 bits, so the result's own rounding dominates; fp32: 3).
template <typename T, int D, int NT, int NQ, int NP>
__global__ void __launch_bounds__(kAttWarps * 32) ds_attend_kernel(const AttendParams p) {
    constexpr int KS = D / 16;       // k-steps of the scores, and row tiles of the output
    constexpr int ROWS = 8 * NT;
    extern __shared__ __align__(16) float sm[];  // [warps][ROWS][D], then [warps][ROWS][4]
    float* sm_o = sm;
    float* sm_r = sm + kAttWarps * ROWS * D;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait();

    // unit = ((sequence [, query token]) * heads + head) * row_groups + row group
    const int64_t unit = blockIdx.x / p.splits;
    const int split = static_cast<int>(blockIdx.x % p.splits);
    const int rg = static_cast<int>(unit % p.row_groups);
    const int h = static_cast<int>(unit / p.row_groups % p.heads);
    const int64_t bq = unit / p.row_groups / p.heads;
    const bool picked = p.indices != nullptr;
    const int64_t b = picked ? bq / p.Q : bq;
    const int q0 = picked ? static_cast<int>(bq % p.Q) : 0;
    const int64_t len = min(static_cast<int64_t>(p.lens[b]), p.max_pos);
    // query token i sees positions below len - (Q - 1 - i)
    const int end_all = static_cast<int>(max(picked ? len - (p.Q - 1 - q0) : len, int64_t(0)));
    const int count = picked ? p.K : end_all;       // positions (or list entries) of this unit
    const int from = split * p.chunk, to = min(from + p.chunk, count);
    if (from >= count && split > 0) return;         // the join reads only splits that have work

    const int32_t* table = p.table + b * p.table_stride;
    const int32_t* list = picked ? p.indices + bq * p.K : nullptr;
    const int page_mask = (1 << p.page_log) - 1;

    // rows of this lane: as key (g) for loading q, as columns (2t, 2t+1) for scores
    const auto row_query = [&](int r, int64_t& off, int& end) -> bool {  // row r of the unit
        if (r >= p.rows) {
            end = 0;
            return false;
        }
        const int qi = picked ? q0 : r / p.group;
        const int hd = h * p.group + (picked ? r : r % p.group);
        off = b * p.q_seq + qi * p.q_tok + hd * p.q_head;
        end = static_cast<int>(max(len - (p.Q - 1 - qi), int64_t(0)));
        return true;
    };
    uint32_t qf[NT][KS][2][NQ];
    float qsum[NT][2];
    int ends[NT][2];
    int first_end = 0x7FFFFFFF;  // below it no row of the CTA masks anything
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        int64_t off = 0;
        int end = 0;
        const bool on = row_query(rg * ROWS + 8 * j + g, off, end);
        const T* q = static_cast<const T*>(p.q) + off + t * (D / 4);
        float sum = 0.f;
#pragma unroll
        for (int kk = 0; kk < KS; ++kk)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int d = 8 * (kk / 2) + 2 * (kk % 2) + half;
                const float x = on ? att_f32(q[d]) : 0.f, y = on ? att_f32(q[d + 4]) : 0.f;
                sum += x + y;
                split_bf16<NQ>(x, y, qf[j][kk][half]);
            }
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
#pragma unroll
        for (int c = 0; c < 2; ++c) {  // rows 2t + c sit in lanes 4 (2t + c)
            qsum[j][c] = __shfl_sync(0xFFFFFFFFu, sum, 4 * (2 * t + c));
            int64_t o2;
            const bool on2 = row_query(rg * ROWS + 8 * j + 2 * t + c, o2, ends[j][c]);
            if (on2) first_end = min(first_end, ends[j][c]);
        }
    }
    first_end = __reduce_min_sync(0xFFFFFFFFu, first_end);

    const auto entry_of = [&](int j, int& pos) -> uint32_t {  // list entry or position j
        pos = 0x7FFFFFFF;
        if (j >= to) return kNoEntry;
        const int at = picked ? list[j] : j;
        if (at < 0 || at >= end_all) return kNoEntry;
        const int page = table[at >> p.page_log];
        if (page < 0 || page >= p.pages) return kNoEntry;
        pos = at;
        return ((static_cast<uint32_t>(page) * p.heads + h) << p.page_log) + (at & page_mask);
    };
    const auto load = [&](AttTile<D>& a, uint32_t entry, int pos) {
        a.pos = pos;
        a.sc = make_uint2(0u, 0u);
        if (entry != kNoEntry) a.sc = reinterpret_cast<const uint2*>(p.scales)[entry];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t e = __shfl_sync(0xFFFFFFFFu, entry, g + 8 * i);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) a.k[i][w] = 0u;
            if (e != kNoEntry) load_words<D / 32>(p.cache + static_cast<uint64_t>(e) * D + t * (D / 8), a.k[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t e = __shfl_sync(0xFFFFFFFFu, entry, 16 * (i >> 2) + 8 * ((i >> 1) & 1) + 2 * t + (i & 1));
#pragma unroll
            for (int w = 0; w < D / 64; ++w) a.v[i][w] = 0u;
            if (e != kNoEntry)
                load_words<D / 64>(p.cache + static_cast<uint64_t>(e) * D + D / 2 + g * (D / 16), a.v[i]);
        }
    };

    float o[NT][KS][4], m[NT][2], l[NT][2], z[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[j][mt][c] = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c) m[j][c] = -INFINITY, l[j][c] = 0.f, z[j][c] = 0.f;
    }
    const float fold = p.scale * kLog2e;

    const auto step = [&](const AttTile<D>& a) {
        // scores of 32 positions: rows of tile i are positions 16 i + {g, g + 8}
        float s[NT][2][4];
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[j][i][c] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                const uint32_t w0 = a.k[2 * i][kk / 2], w1 = a.k[2 * i + 1][kk / 2];
                const int nib = 2 * (kk % 2);
                const uint32_t a0 = codes_bf16(w0, nib), a1 = codes_bf16(w1, nib);
                const uint32_t a2 = codes_bf16(w0, nib + 1), a3 = codes_bf16(w1, nib + 1);
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int n = 0; n < NQ; ++n)
                        mma_bf16(s[j][i], a0, a1, a2, a3, qf[j][kk][0][n], qf[j][kk][1][n]);
            }
        float vs[4], vm[4];
        int pos[4];
        const bool edge = __any_sync(0xFFFFFFFFu, a.pos >= first_end);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t kw = __shfl_sync(0xFFFFFFFFu, a.sc.x, 8 * i + g);
            const uint32_t vw = __shfl_sync(0xFFFFFFFFu, a.sc.y, 8 * i + g);
            pos[i] = __shfl_sync(0xFFFFFFFFu, a.pos, 8 * i + g);
            const float ks = __uint_as_float(kw << 16), km = __uint_as_float(kw & 0xFFFF0000u);
            const float f = ks * fold, base = fmaf(8.f, ks, km) * fold;
            vs[i] = __uint_as_float(vw << 16);
            vm[i] = fmaf(8.f, vs[i], __uint_as_float(vw & 0xFFFF0000u));
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float& x = s[j][i / 2][2 * (i & 1) + c];
                    x = fmaf(x, f, base * qsum[j][c]);
                    if (edge && pos[i] >= ends[j][c]) x = -INFINITY;
                }
        }
        // raise the running maxima where a score passes one by 2^kRaise (or is the first)
        bool up = false;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float x = fmaxf(fmaxf(s[j][0][c], s[j][0][c + 2]), fmaxf(s[j][1][c], s[j][1][c + 2]));
                up |= x > m[j][c] + kRaise;
            }
        if (__any_sync(0xFFFFFFFFu, up)) {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float by[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float x = fmaxf(fmaxf(s[j][0][c], s[j][0][c + 2]), fmaxf(s[j][1][c], s[j][1][c + 2]));
#pragma unroll
                    for (int d = 4; d <= 16; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, d));
                    x = fmaxf(x, m[j][c]);
                    by[c] = x == m[j][c] ? 1.f : exp2_fast(m[j][c] - x);
                    m[j][c] = x;
                    l[j][c] *= by[c];
                    z[j][c] *= by[c];
                }
#pragma unroll
                for (int mt = 0; mt < KS; ++mt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[j][mt][c] *= by[c & 1];
            }
        }
        // weights p, the sums of p and of p (m + 8 s), and p s as the second operand
        uint32_t bf[NT][2][2][NP];  // [row tile][16 positions][first or second 8][part]
#pragma unroll
        for (int j = 0; j < NT; ++j) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float w[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const float x = s[j][i / 2][2 * (i & 1) + c];
                    const bool off = edge && pos[i] >= ends[j][c];
                    const float e = off ? 0.f : exp2_fast(x - m[j][c]);
                    l[j][c] += e;
                    z[j][c] = off ? z[j][c] : fmaf(e, vm[i], z[j][c]);
                    w[c] = off ? 0.f : e * vs[i];
                }
                uint32_t part[NP];
                split_bf16<NP>(w[0], w[1], part);
#pragma unroll
                for (int n = 0; n < NP; ++n) bf[j][i / 2][i & 1][n] = transpose8x8(part[n]);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
                const uint32_t x0 = a.v[4 * i][w], x1 = a.v[4 * i + 1][w];
                const uint32_t y0 = a.v[4 * i + 2][w], y1 = a.v[4 * i + 3][w];
                const uint32_t xl = __byte_perm(x0, x1, 0x5410), xh = __byte_perm(x0, x1, 0x7632);
                const uint32_t yl = __byte_perm(y0, y1, 0x5410), yh = __byte_perm(y0, y1, 0x7632);
#pragma unroll
                for (int n4 = 0; n4 < 4; ++n4) {
                    const uint32_t a0 = codes_bf16(xl, n4), a1 = codes_bf16(xh, n4);
                    const uint32_t a2 = codes_bf16(yl, n4), a3 = codes_bf16(yh, n4);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int n = 0; n < NP; ++n)
                            mma_bf16(o[j][4 * w + n4], a0, a1, a2, a3, bf[j][i][0][n], bf[j][i][1][n]);
                }
            }
    };

    // tiles of this warp: loads of the next tile and the entries of the one after it are in
    // flight while a tile is computed
    constexpr int STRIDE = kAttWarps * kAttTile;
    int j0 = from + warp * kAttTile;
    if (j0 < to) {
        AttTile<D> cur;
        int pos, pos2;
        uint32_t e = entry_of(j0 + lane, pos);
        load(cur, e, pos);
        uint32_t e2 = entry_of(j0 + STRIDE + lane, pos2);
        for (; j0 < to; j0 += STRIDE) {
            AttTile<D> nxt;
            load(nxt, e2, pos2);
            e2 = entry_of(j0 + 2 * STRIDE + lane, pos2);
            step(cur);
            cur = nxt;
        }
    }

    // join the warps: sums over the lanes of a row, then shared memory
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) {
                l[j][c] += __shfl_xor_sync(0xFFFFFFFFu, l[j][c], d);
                z[j][c] += __shfl_xor_sync(0xFFFFFFFFu, z[j][c], d);
            }
            const int r = 8 * j + 2 * t + c;
            if (g == 0) {
                float* q = sm_r + (warp * ROWS + r) * 4;
                q[0] = m[j][c], q[1] = l[j][c], q[2] = z[j][c];
            }
            float* dst = sm_o + (warp * ROWS + r) * D + g * (D / 8);
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
                dst[8 * (mt / 4) + mt % 4] = o[j][mt][c];
                dst[8 * (mt / 4) + mt % 4 + 4] = o[j][mt][c + 2];
            }
        }
    __syncthreads();
    const int rows = min(ROWS, p.rows - rg * ROWS);
    for (int i = tid; i < rows * D; i += kAttWarps * 32) {
        const int r = i / D, d = i % D;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kAttWarps; ++w) top = fmaxf(top, sm_r[(w * ROWS + r) * 4]);
        float acc = 0.f, sum = 0.f;
        if (top > -INFINITY) {
#pragma unroll
            for (int w = 0; w < kAttWarps; ++w) {
                const float* q = sm_r + (w * ROWS + r) * 4;
                const float f = exp2_fast(q[0] - top);
                acc += f * (sm_o[(w * ROWS + r) * D + d] + q[2]);
                sum += f * q[1];
            }
        }
        if (p.splits > 1) {
            const int64_t at = (unit * p.splits + split) * ROWS + r;
            p.ws_o[at * D + d] = acc;
            if (d == 0) {
                p.ws_ml[at * 2] = top;
                p.ws_ml[at * 2 + 1] = sum;
            }
        } else {
            const int ur = rg * ROWS + r;
            const int qi = picked ? q0 : ur / p.group;
            const int hd = h * p.group + (picked ? ur : ur % p.group);
            const int64_t at = (b * p.Q + qi) * (static_cast<int64_t>(p.heads) * p.group) + hd;
            const float y = sum > 0.f ? acc / sum : 0.f;
            if constexpr (sizeof(T) == 2) static_cast<__nv_bfloat16*>(p.out)[at * D + d] = __float2bfloat16_rn(y);
            else static_cast<float*>(p.out)[at * D + d] = y;
            if (d == 0 && p.lse) p.lse[at] = sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
        }
    }
}

// Joins the splits of one query row: one CTA per row, its warps take the splits in turn.
// Only the splits that hold positions are read (the others wrote nothing); their order is
// fixed, so a call's result does not depend on timing.
template <typename T, int D>
__global__ void __launch_bounds__(256) ds_attend_join_kernel(const AttendParams p, int ROWS) {
    __shared__ float sh_o[8][D];
    __shared__ float sh_ml[8][2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    constexpr int PER = D / 32;
    pdl_launch_dependents();
    pdl_wait();
    const int64_t at = blockIdx.x;  // (sequence * Q + token) * query heads + head
    const int hq = p.heads * p.group;
    const int64_t bq = at / hq;
    const int hd = static_cast<int>(at % hq);
    const int64_t b = bq / p.Q;
    const int qi = static_cast<int>(bq % p.Q);
    const bool picked = p.indices != nullptr;
    const int ur = picked ? hd % p.group : qi * p.group + hd % p.group;
    const int64_t unit = ((picked ? bq : b) * p.heads + hd / p.group) * p.row_groups + ur / ROWS;
    const int64_t len = min(static_cast<int64_t>(p.lens[b]), p.max_pos);
    const int64_t count = picked ? p.K : max(len, int64_t(0));
    const int splits = max(1, min(p.splits, static_cast<int>((count + p.chunk - 1) / p.chunk)));
    const int64_t base = unit * p.splits * ROWS + ur % ROWS;
    float top = -INFINITY;
    for (int s = lane; s < splits; s += 32) top = fmaxf(top, p.ws_ml[(base + static_cast<int64_t>(s) * ROWS) * 2]);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    float acc[PER], sum = 0.f;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
    if (top > -INFINITY) {
#pragma unroll 4
        for (int s = warp; s < splits; s += warps) {
            const int64_t e = base + static_cast<int64_t>(s) * ROWS;
            const float f = exp2_fast(p.ws_ml[e * 2] - top);
            sum += f * p.ws_ml[e * 2 + 1];
#pragma unroll
            for (int i = 0; i < PER; ++i) acc[i] += f * p.ws_o[e * D + i * 32 + lane];
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) sh_o[warp][i * 32 + lane] = acc[i];
    if (lane == 0) sh_ml[warp][0] = sum;
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float y = 0.f, total = 0.f;
        for (int w = 0; w < warps; ++w) y += sh_o[w][d], total += sh_ml[w][0];
        y = total > 0.f ? y / total : 0.f;
        if constexpr (sizeof(T) == 2) static_cast<__nv_bfloat16*>(p.out)[at * D + d] = __float2bfloat16_rn(y);
        else static_cast<float*>(p.out)[at * D + d] = y;
        if (d == 0 && p.lse) p.lse[at] = total > 0.f ? (top + log2f(total)) * kLn2 : -INFINITY;
    }
}

template <typename T, int D, int NT>
static ds_status attend(const AttendParams& p, int64_t units, int64_t out_rows, cudaStream_t stream) {
    constexpr int NQ = sizeof(T) == 2 ? 1 : 3, NP = sizeof(T) == 2 ? 2 : 3;
    auto kern = ds_attend_kernel<T, D, NT, NQ, NP>;
    const size_t smem = static_cast<size_t>(kAttWarps) * 8 * NT * (D + 4) * sizeof(float);
    if (smem > 48 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return DS_ERR_CUDA;
    const dim3 grid(static_cast<unsigned>(units * p.splits));
    const ds_status st = launch_pdl(kern, grid, kAttWarps * 32, smem, 1, stream, p);
    if (st != DS_OK || p.splits == 1) return st;
    int warps = 1;
    while (warps < 8 && warps < p.splits) warps <<= 1;
    return launch_pdl(ds_attend_join_kernel<T, D>, dim3(static_cast<unsigned>(out_rows)), warps * 32, 0, 1, stream, p,
                      8 * NT);
}

template <typename T, int D>
static ds_status attend_rows(const AttendParams& p, int nt, int64_t units, int64_t out_rows, cudaStream_t stream) {
    if (nt == 1) return attend<T, D, 1>(p, units, out_rows, stream);
    return attend<T, D, 2>(p, units, out_rows, stream);
}

}  // namespace dsk

using namespace dsk;

extern "C" {

ds_status ds_cache_attention(const void* q, int32_t dtype, int64_t sequences, int32_t tokens, int32_t q_heads,
                             int32_t D, int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride,
                             const void* cache, const void* scales, int64_t pages, int32_t heads, int32_t page,
                             const int32_t* table, int64_t table_width, int64_t table_stride, const int32_t* lens,
                             const int32_t* indices, int32_t K, float scale, void* out, float* out_lse,
                             cudaStream_t stream) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || sequences < 0 || tokens < 1 || q_heads < 1 || heads < 1 ||
        q_heads % heads != 0 || pages < 1 || page < 1 || table_width < 1 || table_stride < table_width || K < 0)
        return DS_ERR_INVALID_ARG;
    if (q_seq_stride < 0 || q_token_stride < 0 || q_head_stride < 0 || !isfinite(scale)) return DS_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || (page & (page - 1)) != 0) return DS_ERR_UNSUPPORTED;
    if (pages * page * heads >= 0xFFFFFFFFLL || pages > 0x7FFFFFFFLL || table_width > (int64_t(1) << 30) / page)
        return DS_ERR_UNSUPPORTED;
    if (sequences == 0) return DS_OK;
    if (!q || !cache || !scales || !table || !lens || !out || (K > 0 && !indices)) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    if (!aligned16(cache) || reinterpret_cast<uintptr_t>(scales) % 8 || reinterpret_cast<uintptr_t>(q) % es ||
        reinterpret_cast<uintptr_t>(out) % es)
        return DS_ERR_ALIGNMENT;
    const void* words[] = {table, lens, indices, out_lse};
    for (const void* w : words)
        if (reinterpret_cast<uintptr_t>(w) % 4) return DS_ERR_ALIGNMENT;
    int dev = 0;
    DevInfo info;
    if (cudaGetDevice(&dev) != cudaSuccess || !dev_info(dev, info)) return DS_ERR_CUDA;

    AttendParams p = {};
    p.q = q;
    p.q_seq = q_seq_stride;
    p.q_tok = q_token_stride;
    p.q_head = q_head_stride;
    p.cache = static_cast<const uint8_t*>(cache);
    p.scales = static_cast<const uint32_t*>(scales);
    p.table = table;
    p.table_stride = table_stride;
    p.lens = lens;
    p.indices = indices;
    p.out = out;
    p.lse = out_lse;
    p.max_pos = table_width * page;
    p.Q = tokens;
    p.K = K;
    p.heads = heads;
    p.group = q_heads / heads;
    while ((1 << p.page_log) < page) ++p.page_log;
    p.pages = static_cast<int32_t>(pages);
    p.scale = scale;
    const int64_t rows = indices ? p.group : static_cast<int64_t>(p.group) * tokens;
    if (rows > (1 << 20)) return DS_ERR_UNSUPPORTED;
    p.rows = static_cast<int32_t>(rows);
    const int nt = rows > 8 ? 2 : 1;
    p.row_groups = (p.rows + 8 * nt - 1) / (8 * nt);
    const int64_t units = (indices ? sequences * tokens : sequences) * heads * p.row_groups;
    const int64_t out_rows = sequences * tokens * q_heads;
    // splits: enough CTAs for several per SM, at least four tiles for each warp
    const int64_t span = indices ? K : p.max_pos;
    const int64_t unit_tiles = kAttWarps * kAttTile;
    int64_t splits = (static_cast<int64_t>(info.sms) * 8 + units - 1) / units;
    const int64_t most = (span + 2 * unit_tiles - 1) / (2 * unit_tiles);
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
    int64_t chunk = (span + splits - 1) / splits;
    chunk = (chunk + unit_tiles - 1) / unit_tiles * unit_tiles;
    if (chunk < unit_tiles) chunk = unit_tiles;
    splits = (span + chunk - 1) / chunk;
    if (splits < 1) splits = 1;
    p.splits = static_cast<int32_t>(splits);
    p.chunk = static_cast<int32_t>(chunk);
    if (units * splits > 0x7FFFFFFFLL || out_rows > 0x7FFFFFFFLL) return DS_ERR_UNSUPPORTED;
    if (splits > 1) {
        const size_t entries = static_cast<size_t>(units) * splits * 8 * nt;
        void* ws = nullptr;
        const ds_status st = library_workspace(dev, kWsAttend, entries * (D + 2) * sizeof(float), stream, &ws);
        if (st != DS_OK) return st;
        p.ws_o = static_cast<float*>(ws);
        p.ws_ml = p.ws_o + entries * D;
    }
    if (dtype == DS_BF16)
        return D == 64 ? attend_rows<__nv_bfloat16, 64>(p, nt, units, out_rows, stream)
                       : attend_rows<__nv_bfloat16, 128>(p, nt, units, out_rows, stream);
    return D == 64 ? attend_rows<float, 64>(p, nt, units, out_rows, stream)
                   : attend_rows<float, 128>(p, nt, units, out_rows, stream);
}

}  // extern "C"
