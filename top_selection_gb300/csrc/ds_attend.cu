// ds_attend.cu -- attention of new tokens over a paged cache of 4-bit keys and values
// (ds_cache_attention): every position of the context, or the positions a top-k selected.
//
// A key row of the cache stands for s c + m (codes c, bf16 scale s and minimum m, see
// ds_cache.cu), so a query row q scores it as
//     q . (s c + m) = s (q . c) + m (sum q).
// With weights p and w = f16(p s) (times a power of two), the values add up to
//     sum p (s c + m) = sum w (c - 7.5)  +  sum p (m + 7.5 s).
// The first sum is taken as  sum_even w c - sum_odd w (15 - c) - 7.5 (sum_even w - sum_odd w)  over
// even and odd positions (complementing a word of codes is one instruction): the running sums stay
// near zero where weights are alike, and the rounding of w and of the matrix unit's additions
// (which cut off) then do not pile up against a result that averages out.  Over 4 x 1M positions the
// error was 2.5 times bf16's own rounding with plain codes; this way it adds nothing to it.
// sum_even w - sum_odd w comes from the matrix unit as well, against a row of ones.
//
// The codes never leave registers once they are there: with tokens as the rows of the matrix
// instruction, the four lanes that share a fragment row read a token's codes as they lie in
// memory (any order of the contracted dimension serves, as long as q is read in the same
// order).  A masked word is the operand: the 16-bit pattern c, or 16 c, is the subnormal f16
// number c 2^-24, or 16 c 2^-24, and the powers of two are taken out of q beforehand and out of
// the sums at the end.  Eight codes cost five instructions (one shift, four ANDs; value words of
// two tokens are interleaved first), against eleven for conversion by an offset.  The matrix unit
// keeps fewer bits of subnormal products, far below bf16's rounding; fp32 takes normal numbers.
//
// m16n8k16 (mma.sync) rather than tcgen05: with up to 16 query rows per key head the operand that
// streams is the cache, and tcgen05 takes it from shared memory only, so each tile would be
// expanded to twice its bytes or more, stored and read back.  Here the cache's bytes are the
// operand.  More rows go in groups of 16, each of which reads and masks the cache again: 4 x 1M positions
// with 16 rows 132 us, with 64 rows 476 (fp32 235 and 883).  There one expansion for all rows would
// serve tcgen05, which has not been tried.
//
// Rows: the query rows that share a key head (heads of a group, and for whole contexts the
// tokens of the step as well) in tiles of 8; a CTA takes up to 8 * NT of them and one split of
// the positions; its warps take tiles of 32 positions in turn, each through its own ring of
// asynchronous copies.  Softmax runs online per warp: one running maximum per row, raised only
// when a score passes it by 2^kRaise, sums per lane.  Warps are joined in shared memory, splits
// over a cluster's or by a second kernel.
//
// 16 rows are bound by the matrix, ALU and FMA pipes together (4 x 1M positions, 570 MB: 132 us, 4.3
// TB/s, matrix pipe 48 %), 8 rows nearly by memory (100 us, 5.7 TB/s), short contexts by the chain from
// lengths over pages and codes to the join (one of 4096 positions, 8 heads: 9.8 us).  fp32 queries take
// twice the matrix instructions, and each sum's additions outside of them (16 rows 235 us, 8 rows 164).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "ds_common.cuh"
#include "ds_host.cuh"
#include "ds_topk.h"

namespace dsk {

constexpr int kAttWarps = 4;                   // warps of a CTA, or one where there are many units
constexpr int kAttTile = 32;                   // positions per warp and step
constexpr int kAttStages = 3;                  // tiles of a warp's ring
constexpr int kAttCluster = 8;                 // portable cluster size
constexpr uint32_t kNoEntry = 0xFFFFFFFFu;
constexpr int kNoPosition = 0x7FFFFFFF;        // of a place without an entry
constexpr uint32_t kAll = 0xFFFFFFFFu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNone = -3e38f;                // below any score: running maximum of a row that has seen nothing
// Weights as f16: p is at most 2^kRaise, and w = p s kTop / r, r a power of two near the largest
// value scale |s| seen and never below an eighth of one (a row of values whose minimum bf16 rounds up
// past its maximum has s < 0).  The largest |w| is 16 * 8 * 256 = 2^15
// (f16 ends at 2^16), and the heaviest position's is about 2^8, 22 binades above the subnormals.
constexpr float kRaise = 4.0f, kTop = 256.0f, kOver = 2048.0f;

struct AttendParams {
    const void* q;
    int64_t q_seq, q_tok, q_head;  // element strides
    const uint8_t* cache;
    const uint2* scales;           // per entry: key (s, m), value (s, m)
    const int32_t* table;
    int64_t table_stride;
    const int32_t* lens;
    const int32_t* indices;        // [B, Q, K] or null
    void* out;
    float* lse;
    float4* ws_o;                  // splits' partial results, one a CTA: [CTA][fragment][lane]
    float2* ws_ml;                 //                                     [CTA][rows]: maximum, sum of weights
    int2* ws_cut;                  // fitted splits: each unit's first CTA and number of splits
    int32_t max_pos, span;         // table width * page; max_pos or K
    int32_t Q, K, heads, group, page_log, pages;
    int32_t rows;                  // query rows per unit before tiling
    int32_t row_groups, splits, chunk;
    int32_t q_vec;                 // q rows start on 16 bytes
    int32_t cluster;               // the splits of a unit are one cluster and join in it
    int32_t sequences;
    int32_t fit;                   // > 0: splits by length (`fitted`), so many a head and row group
    float scale;
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float2 unpack_f16(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

// (a, b) = the sum of NS pairs of f16 (11 bits each)
template <int NS>
__device__ __forceinline__ void split_f16(float a, float b, uint32_t (&part)[NS]) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
        part[i] = pack_f16(a, b);
        if (i + 1 < NS) {
            const float2 f = unpack_f16(part[i]);
            a -= f.x;
            b -= f.y;
        }
    }
}

// Codes `nib` (0 .. 3) of both halves of w (w already moved down by 8 for nib >= 2): two f16
// numbers c 2^-24, for odd nib 16 c 2^-24.  CENTRE: c - 8 and 16 (c - 8), by way of 1024 + c (normal
// numbers: the matrix unit keeps fewer bits of subnormal ones' products, 9e-6 of an fp32 result).
template <bool CENTRE>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int nib) {
    const uint32_t mask = nib & 1 ? 0x00F000F0u : 0x000F000Fu;
    if (!CENTRE) return w & mask;
    const uint32_t x = (w & mask) | 0x64006400u, mid = nib & 1 ? 0x64806480u : 0x64086408u;
    const __half2 r = __hsub2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&mid));
    return *reinterpret_cast<const uint32_t*>(&r);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
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

// two fp32 numbers to an instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
// four results times f, in the output's type
__device__ __forceinline__ void store4(float* p, float4 v, float f) {
    *reinterpret_cast<float4*>(p) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v, float f) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * f, v.y * f), b = __floats2bfloat162_rn(v.z * f, v.w * f);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
template <typename T>
__device__ __forceinline__ T to_type(float v) {
    if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
    else return v;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// asynchronous copies global -> shared; `on` false fills the bytes with zeros
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool on) {
    const int n = on ? BYTES : 0;
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
// 16 bytes at `at` bytes behind both addresses
template <int AT>
__device__ __forceinline__ void copy_async_at(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;" ::"r"(dst), "l"(src), "n"(AT) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A tile in shared memory: 32 rows of D bytes (key codes, value codes) and their scales.
// 16-byte pieces of a row are permuted so that the reads of a warp meet every
// bank once: a key read takes 8 rows by the lanes' quarter, a value read rows 2t apart.
template <int D>
struct TileAt {
    static constexpr int kRowBytes = D;
    static constexpr int kScaleAt = kAttTile * D;
    static constexpr int kBytes = kScaleAt + kAttTile * 8;
    static __device__ __forceinline__ int piece(int row, int chunk) {
        const int x = D == 128 ? (((row >> 1) & 3) << 1) ^ ((row & 1) << 2) : ((row >> 1) & 1) << 1;
        return row * D + ((chunk ^ x) << 4);
    }
};

// Writes joined output fragments of a unit, divided by the sums of the weights, and lse.
template <typename T, int D>
struct Emit {
    const AttendParams& p;
    int b, h, q0;
    bool picked;
    int first, rows, g, t;  // the row group's first row and its rows; the lane's place
    __device__ __forceinline__ int64_t row_of(int r) const {  // row r of the group in the output
        const int ur = first + r;
        const int qi = picked ? q0 : ur / p.group;
        const int hd = h * p.group + (picked ? ur : ur - qi * p.group);
        return (static_cast<int64_t>(b) * p.Q + qi) * (static_cast<int64_t>(p.heads) * p.group) + hd;
    }
    __device__ __forceinline__ void lse(int64_t e, float top, float sum) const {
        if (p.lse) p.lse[e] = sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
    }
    // the four fragments of row tile and code word `item`: numbers 8 w .. 8 w + 7 of the lane's eighth
    __device__ __forceinline__ void four(int item, const float4 (&a)[4], float top0, float sum0, float top1,
                                         float sum1) const {
        const int j = item / (D / 64), w = item % (D / 64), r = 8 * j + 2 * t;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (r + c >= rows) continue;
            const int64_t e = row_of(r + c);
            const float sum = c ? sum1 : sum0, f = sum > 0.f ? 1.f / sum : 0.f;
            T* dst = static_cast<T*>(p.out) + e * D + g * (D / 8) + 8 * w;
            store4(dst, c ? make_float4(a[0].y, a[1].y, a[2].y, a[3].y) : make_float4(a[0].x, a[1].x, a[2].x, a[3].x), f);
            store4(dst + 4, c ? make_float4(a[0].w, a[1].w, a[2].w, a[3].w) : make_float4(a[0].z, a[1].z, a[2].z, a[3].z), f);
            if (g == 0 && w == 0) lse(e, c ? top1 : top0, sum);
        }
    }
    // one fragment: numbers k and k + 4 of a word
    __device__ __forceinline__ void one(int frag, float4 a, float top0, float sum0, float top1, float sum1) const {
        const int j = frag / (D / 16), mt = frag % (D / 16), r = 8 * j + 2 * t;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (r + c >= rows) continue;
            const int64_t e = row_of(r + c);
            const float sum = c ? sum1 : sum0, f = sum > 0.f ? 1.f / sum : 0.f;
            T* dst = static_cast<T*>(p.out) + e * D + g * (D / 8) + 8 * (mt / 4) + mt % 4;
            dst[0] = to_type<T>((c ? a.y : a.x) * f);
            dst[4] = to_type<T>((c ? a.w : a.z) * f);
            if (g == 0 && mt == 0) lse(e, c ? top1 : top0, sum);
        }
    }
};

// CTAs per SM that the registers are cut for: 8 warps for 16 rows, 12 for 8
constexpr int att_resident(int NT, int WARPS) {
    return (NT == 1 ? 12 : 8) / WARPS;
}

// Splits by the contexts' lengths, which the host does not know: all of one size, the smallest of 32
// for which the places that run at once are enough (p.fit for each head and row group).  Every warp
// finds its CTA's split by itself, by the same arithmetic.
struct Fitted {
    uint32_t unit;
    int split, splits;  // splits 0: this CTA has none
    int steps, first;   // of STEP positions in a split; the unit's first CTA
};
template <int STEP>
__device__ __forceinline__ Fitted fitted(const AttendParams& p, int lane) {
    const auto steps_of = [&](int b) { return (max(min(p.lens[b], p.max_pos), 1) + STEP - 1) / STEP; };
    // ceil(n / c): the product is at least 1 / 2 c from a whole number, more than its error
    const auto splits_of = [](int n, float by) { return static_cast<int>((static_cast<float>(n) - 0.5f) * by) + 1; };
    int64_t sum = 0;
#pragma unroll 4
    for (int i = lane; i < p.sequences; i += 32) sum += steps_of(i);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
    // lane l: 1 + l / 16 times the size that fills every place; the last ones' splits always fit, as
    // half of the places are enough for all sequences' first
    const int least = static_cast<int>((sum + p.fit - 1) / p.fit);
    const int mine = least + (least * lane + 15) / 16;
    float by = 1.f / static_cast<float>(mine);
    int need = 0;
#pragma unroll 4
    for (int i = 0; i < p.sequences; ++i) need += splits_of(steps_of(i), by);
    const int best = __ffs(__ballot_sync(kAll, need <= p.fit)) - 1;
    Fitted f = {0u, 0, 0, __shfl_sync(kAll, mine, best), 0};
    by = __shfl_sync(kAll, by, best);
    const int per = p.heads * p.row_groups, rank = static_cast<int>(blockIdx.x) / per, place = static_cast<int>(blockIdx.x) - rank * per;
    int before = 0;
    for (int i = 0; i < p.sequences; i += 32) {
        const int n = i + lane < p.sequences ? splits_of(steps_of(i + lane), by) : 0;
        int upto = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int x = __shfl_up_sync(kAll, upto, d);
            if (lane >= d) upto += x;
        }
        const uint32_t behind = __ballot_sync(kAll, before + upto > rank);
        if (behind) {
            const int at = __ffs(behind) - 1;
            f.splits = __shfl_sync(kAll, n, at);
            const int start = before + __shfl_sync(kAll, upto, at) - f.splits;
            f.split = rank - start;
            f.unit = static_cast<uint32_t>(i + at) * per + place;
            f.first = start * per + place;
            break;
        }
        before += __shfl_sync(kAll, upto, 31);
    }
    return f;
}

// T: type of q and out.  NQ / NP: f16 parts of q and of the weights.  bf16: one part each (q is
// exact, a weight keeps 11 bits, and the result's rounding to 8 dominates); fp32: two, 22 bits,
// and the codes centred, so that sums cancel less.
// TOKENS: the rows are of several tokens, which see different positions.
template <typename T, int D, int NT, int NQ, int NP, int WARPS, bool TOKENS>
__global__ void __launch_bounds__(WARPS * 32, att_resident(NT, WARPS)) ds_attend_kernel(const AttendParams p) {
    constexpr int KS = D / 16;       // k-steps of the scores, and row tiles of the output
    constexpr int ROWS = 8 * NT;
    constexpr bool CENTRE = sizeof(T) == 4;
    // fp32: the matrix unit's additions cut off, so each of its sums starts at zero and is added here
    constexpr bool EXACT = sizeof(T) == 4;
    constexpr float MID = CENTRE ? 8.f : 7.5f;
    constexpr float kUnit = CENTRE ? 1.f : 16777216.f;  // an operand's code counts 1 / kUnit
    using At = TileAt<D>;
    extern __shared__ __align__(128) unsigned char smem[];  // the warps' rings; then the join
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait();

    // unit = ((sequence [, query token]) * heads + head) * row_groups + row group
    constexpr int STRIDE = WARPS * kAttTile;
    uint32_t unit;
    int split, splits = p.splits, chunk = p.chunk;
    if (p.fit > 0) {
        const Fitted f = fitted<STRIDE>(p, lane);
        if (f.splits == 0) return;
        if (f.split == 0 && tid == 0) p.ws_cut[f.unit] = make_int2(f.first, f.splits);
        unit = f.unit;
        split = f.split;
        splits = f.splits;
        chunk = f.steps * STRIDE;
    } else {
        unit = blockIdx.x / static_cast<uint32_t>(splits);
        split = static_cast<int>(blockIdx.x - unit * splits);
    }
    const uint32_t uh = unit / static_cast<uint32_t>(p.row_groups);
    const int rg = static_cast<int>(unit - uh * p.row_groups);
    const int bq = static_cast<int>(uh / static_cast<uint32_t>(p.heads));
    const int h = static_cast<int>(uh - bq * p.heads);
    const bool picked = p.indices != nullptr;
    const int b = picked ? bq / p.Q : bq;
    const int q0 = picked ? bq % p.Q : 0;
    const int length = p.lens[b];
    const int from = split * chunk;
    const int32_t* table = p.table + b * p.table_stride;
    const int32_t* list = picked ? p.indices + static_cast<int64_t>(bq) * p.K : nullptr;
    const int page_mask = (1 << p.page_log) - 1;

    // Entries come in three steps, so that no load waits for another: the position at place j (a
    // list's value), its page, and the entry, each a tile ahead of the next.  Loads are made in
    // range whatever the values are (a list's and a table's are the caller's); the entry decides.
    const int last = min(from + chunk, p.span);
    const auto position_at = [&](int j) -> int { return j >= last ? -1 : picked ? list[j] : j; };
    const auto page_of = [&](int at) -> int {
        return table[(static_cast<uint32_t>(at) < static_cast<uint32_t>(p.max_pos) ? at : 0) >> p.page_log];
    };
    // tiles of this warp: two in flight while one is computed
    int j0 = from + warp * kAttTile;
    int ahead[kAttStages], page[kAttStages];
#pragma unroll
    for (int s = 0; s < kAttStages; ++s) ahead[s] = position_at(j0 + s * STRIDE + lane);
    int at_far = position_at(j0 + kAttStages * STRIDE + lane);
#pragma unroll
    for (int s = 0; s < kAttStages; ++s) page[s] = page_of(ahead[s]);

    // the length comes beside the first pages, not before them
    const int len = max(min(length, p.max_pos), 0);
    // query token i sees positions below len - (Q - 1 - i)
    const int end_all = max(picked ? len - (p.Q - 1 - q0) : len, 0);
    const int count = picked ? p.K : end_all;       // positions (or list entries) of this unit
    const int to = min(from + chunk, count);
    // without a cluster the join is a kernel, which reads only splits that have work
    if (!p.cluster && from >= count && split > 0) return;

    const auto entry_of = [&](int at, int page, int& pos) -> uint32_t {
        const bool seen = at >= 0 && at < end_all && static_cast<uint32_t>(page) < static_cast<uint32_t>(p.pages);
        pos = seen ? at : kNoPosition;
        return seen ? ((static_cast<uint32_t>(page) * p.heads + h) << p.page_log) + (at & page_mask) : kNoEntry;
    };
    unsigned char* ring = smem + warp * (kAttStages * At::kBytes);
    const uint32_t ring_at = smem_u32(ring);
    // Copies a tile into a slot of the ring.  Positions that share a page lie side by side, so a
    // whole tile of them is one run of 32 D bytes; else each row goes by its own entry.
    constexpr int CH = D / 16, PER = 32 / CH;  // 16-byte pieces of a row; rows per instruction
    const int row0 = lane / CH, ch = lane % CH;
    const auto issue = [&](int slot, uint32_t entry, bool run) {
        const uint32_t base = ring_at + slot * At::kBytes;
        if (run) {
            const uint8_t* src = p.cache + static_cast<uint64_t>(entry) * D - (lane * D - lane * 16);
            // the permutation of a row's pieces repeats every 8 rows, two (D = 64: one) copies
            const uint32_t d0 = base + At::piece(row0, ch), d1 = base + At::piece(PER + row0, ch) - 512;
            copy_async_at<0>(d0, src);
            copy_async_at<512>(d1, src);
            copy_async_at<2 * 512>(d0, src);
            copy_async_at<3 * 512>(d1, src);
            if constexpr (D == 128) {
                copy_async_at<4 * 512>(d0, src);
                copy_async_at<5 * 512>(d1, src);
                copy_async_at<6 * 512>(d0, src);
                copy_async_at<7 * 512>(d1, src);
            }
        } else {
#pragma unroll
            for (int i = 0; i < kAttTile / PER; ++i) {
                const uint32_t e = __shfl_sync(kAll, entry, i * PER + row0);
                const uint8_t* src = p.cache + (e == kNoEntry ? 0 : static_cast<uint64_t>(e) * D) + ch * 16;
                copy_async<16>(base + At::piece(i * PER + row0, ch), src, e != kNoEntry);
            }
        }
        copy_async<8>(base + At::kScaleAt + lane * 8, p.scales + (entry == kNoEntry ? 0u : entry), entry != kNoEntry);
        copies_commit();
    };
    // a tile of consecutive positions inside one page, none of them missing
    const bool runs = !picked && p.page_log >= 5;
    const auto is_run = [&](uint32_t entry) { return runs && __all_sync(kAll, entry != kNoEntry); };

    int pos[kAttStages];  // the lane's position in each tile: current, in flight, next
#pragma unroll
    for (int s = 0; s + 1 < kAttStages; ++s) {
        const uint32_t entry = entry_of(ahead[s], page[s], pos[s]);
        issue(s, entry, is_run(entry));
    }
    int at_ahead = ahead[kAttStages - 1], page_ahead = page[kAttStages - 1];

    // q as the second operand: row g of each tile, the lane's quarter of the numbers in the
    // order of the codes, times a power of two that brings the row's largest to 2^13 .. 2^14, and
    // another 1/16 against codes that count 16-fold.  Each row has its own: under one for all of them
    // a row 2^22 below the largest loses bits to f16's range, and a padded token's row may hold
    // anything.
    const auto row_query = [&](int r, int64_t& off, int& end) -> bool {  // row r of the unit
        if (r >= p.rows) {
            end = 0;
            return false;
        }
        const int qi = picked ? q0 : r / p.group;
        const int hd = h * p.group + (picked ? r : r - qi * p.group);
        off = b * p.q_seq + qi * p.q_tok + hd * p.q_head;
        end = max(len - (p.Q - 1 - qi), 0);
        return true;
    };
    constexpr int QW = 2 * NT * NQ;  // words of a lane and k-step: kept in shared memory
    uint32_t* sm_q = reinterpret_cast<uint32_t*>(smem + WARPS * kAttStages * At::kBytes);
    float2 qsum[NT];
    int ends[NT][2];
    int first_end = 0x7FFFFFFF;  // below it no row of the CTA masks anything
    float2 fold[NT];  // what a score of codes and operand counts, of rows 2t and 2t + 1
    {
        float x[NT][D / 4], by[NT];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            int64_t off = 0;
            int end = 0;
            const bool on = row_query(rg * ROWS + 8 * j + g, off, end);
            const T* q = static_cast<const T*>(p.q) + off + t * (D / 4);
            if (p.q_vec) {
                constexpr int PER = 16 / sizeof(T);
#pragma unroll
                for (int i = 0; i < D / 4 / PER; ++i) {
                    const uint4 w = on ? reinterpret_cast<const uint4*>(q)[i] : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if constexpr (sizeof(T) == 2) {
                            x[j][i * PER + 2 * k] = __uint_as_float(u[k] << 16);
                            x[j][i * PER + 2 * k + 1] = __uint_as_float(u[k] & 0xFFFF0000u);
                        } else {
                            x[j][i * PER + k] = __uint_as_float(u[k]);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < D / 4; ++i) x[j][i] = on ? static_cast<float>(q[i]) : 0.f;
            }
            float sum = 0.f, top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 4; ++i) {
                sum += x[j][i];
                const float a = fabsf(x[j][i]);
                top = fmaxf(top, a < INFINITY ? a : 0.f);
            }
            sum += __shfl_xor_sync(kAll, sum, 1);
            sum += __shfl_xor_sync(kAll, sum, 2);
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
            const int e = static_cast<int>(__float_as_uint(top) >> 23);  // biased exponent
            const int up = e == 0 ? 0 : min(max(13 - (e - 127), -100), 100);
            by[j] = __uint_as_float(static_cast<uint32_t>(up + 127) << 23);
            const float down = p.scale * kLog2e * kUnit * __uint_as_float(static_cast<uint32_t>(127 - up) << 23);
            sum *= p.scale * kLog2e;
            // rows 2t + c sit in lanes 4 (2t + c)
            qsum[j] = make_float2(__shfl_sync(kAll, sum, 8 * t), __shfl_sync(kAll, sum, 8 * t + 4));
            fold[j] = make_float2(__shfl_sync(kAll, down, 8 * t), __shfl_sync(kAll, down, 8 * t + 4));
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                int64_t o2;
                const bool on2 = row_query(rg * ROWS + 8 * j + 2 * t + c, o2, ends[j][c]);
                if (on2) first_end = min(first_end, ends[j][c]);
            }
        }
        first_end = __reduce_min_sync(kAll, first_end);
        // each warp writes its share of the k-steps
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            if (kk % WARPS != warp) continue;
            uint32_t w[QW];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int d = 8 * (kk / 2) + 2 * (kk % 2) + half;
                    const float f = half ? by[j] * 0.0625f : by[j];
                    uint32_t part[NQ];
                    split_f16<NQ>(x[j][d] * f, x[j][d + 4] * f, part);
#pragma unroll
                    for (int n = 0; n < NQ; ++n) w[(j * NQ + n) * 2 + half] = part[n];
                }
#pragma unroll
            for (int i = 0; i < QW / 2; ++i)
                reinterpret_cast<uint2*>(sm_q)[(kk * 32 + lane) * (QW / 2) + i] = make_uint2(w[2 * i], w[2 * i + 1]);
        }
    }

    __syncthreads();
    float o[NT][KS][4], ones[NT][4];
    float2 neg_m[NT], l[NT], z[NT];  // minus the running maximum, sums of p and p (m + MID s)
    uint32_t unseen = 0u;            // rows of this lane without a score so far
    bool fresh = true;               // the warp has such a row
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
        for (int mt = 0; mt < KS; ++mt)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[j][mt][c] = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) ones[j][c] = 0.f;
        neg_m[j] = l[j] = z[j] = both(0.f);
        const int r = rg * ROWS + 8 * j + 2 * t;
        unseen |= (r < p.rows ? 1u : 0u) << (2 * j) | (r + 1 < p.rows ? 2u : 0u) << (2 * j);
    }
    float wmul = 1.2676506e30f;  // kTop / r; 2^100 until a value scale has been seen
    const float sign = !CENTRE && (g & 1) ? -1.f : 1.f;  // of the weights of this lane's positions

    int slot = 0;
    // the least end behind position x, and the last
    const auto end_past = [&](int x) -> int {
        int e = kNoPosition;
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c)
                if (ends[j][c] > x) e = min(e, ends[j][c]);
        return __reduce_min_sync(kAll, e);
    };
    const auto last_end = [&]() -> int {
        int e = 0;
#pragma unroll
        for (int j = 0; j < NT; ++j) e = max(e, max(ends[j][0], ends[j][1]));
        return __reduce_max_sync(kAll, e);
    };
    // The tiles in turn, in one run as a rule.  TOKENS: a scale that some row does not see (an unwritten slot
    // behind a padded draft may hold anything) must not set r while that row's weights are rounded.
    // A tile where it is more than 8 times the largest that the tile's rows all see ends the run: it
    // is worked through for the positions that they all see, then again for each further one, upwards.  Rows
    // that do not see it have no weights left then, and what they have summed moves by a power of two
    // and back.  The state of such turns lies in shared memory, since registers are short: the first
    // position behind the present one, 0 for an ordinary run, and the end of the split.  (Rows of one token
    // have a kernel without all this, which takes 2 % of a long context's time, 5 % for fp32.)
    volatile int* turn = reinterpret_cast<int*>(smem + WARPS * kAttStages * At::kBytes + KS * 32 * QW * 4) + 2 * warp;
    if (TOKENS && lane == 0) turn[0] = 0;
    int upto = to;
    while (true) {
        for (; j0 < upto; j0 += STRIDE) {
            copies_wait<kAttStages - 2>();
            __syncwarp();
            {
                int next = slot + kAttStages - 1;
                if (next >= kAttStages) next -= kAttStages;
                const uint32_t entry = entry_of(at_ahead, page_ahead, pos[kAttStages - 1]);
                issue(next, entry, is_run(entry));
            }
            int here = pos[0];
#pragma unroll
            for (int i = 0; i + 1 < kAttStages; ++i) pos[i] = pos[i + 1];
            at_ahead = at_far;
            page_ahead = page_of(at_ahead);
            at_far = position_at(j0 + (kAttStages + 1) * STRIDE + lane);
            const unsigned char* tile = ring + slot * At::kBytes;
            if (++slot == kAttStages) slot = 0;

            // scores of 32 positions: rows of tile i are positions 16 i + {g, g + 8}
            float s[NT][2][4];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[j][i][c] = 0.f;
            uint32_t kw[4][D / 32];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 8 * r + g;
                if constexpr (D == 128) {
                    const uint4 w = *reinterpret_cast<const uint4*>(tile + At::piece(row, t));
                    kw[r][0] = w.x, kw[r][1] = w.y, kw[r][2] = w.z, kw[r][3] = w.w;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(tile + At::piece(row, t >> 1) + 8 * (t & 1));
                    kw[r][0] = w.x, kw[r][1] = w.y;
                }
            }
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                const int sh = 8 * (kk & 1);
                uint32_t qf[QW];
                if constexpr (QW == 2) {
                    const uint2 w = reinterpret_cast<const uint2*>(sm_q)[kk * 32 + lane];
                    qf[0] = w.x, qf[1] = w.y;
                } else {
#pragma unroll
                    for (int i = 0; i < QW / 4; ++i) {
                        const uint4 w = reinterpret_cast<const uint4*>(sm_q)[(kk * 32 + lane) * (QW / 4) + i];
                        qf[4 * i] = w.x, qf[4 * i + 1] = w.y, qf[4 * i + 2] = w.z, qf[4 * i + 3] = w.w;
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t w0 = kw[2 * i][kk / 2] >> sh, w1 = kw[2 * i + 1][kk / 2] >> sh;
                    const uint32_t a0 = code_pair<CENTRE>(w0, 0), a1 = code_pair<CENTRE>(w1, 0);
                    const uint32_t a2 = code_pair<CENTRE>(w0, 1), a3 = code_pair<CENTRE>(w1, 1);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        float step[4] = {0.f, 0.f, 0.f, 0.f};
                        float(&sum)[4] = EXACT ? step : s[j][i];
#pragma unroll
                        for (int n = NQ - 1; n >= 0; --n)
                            mma_f16(sum, a0, a1, a2, a3, qf[(j * NQ + n) * 2], qf[(j * NQ + n) * 2 + 1]);
                        if (EXACT) {
#pragma unroll
                            for (int c = 0; c < 4; ++c) s[j][i][c] += step[c];
                        }
                    }
                }
            }
            float vs[4], vm[4];
            int at[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint2 sc = *reinterpret_cast<const uint2*>(tile + At::kScaleAt + (8 * i + g) * 8);
                const float ks = __uint_as_float(sc.x << 16), km = __uint_as_float(sc.x & 0xFFFF0000u);
                vs[i] = __uint_as_float(sc.y << 16);
                vm[i] = fmaf(MID, vs[i], __uint_as_float(sc.y & 0xFFFF0000u));
                const float2 ks2 = both(ks), base = both(CENTRE ? fmaf(8.f, ks, km) : km);
#pragma unroll
                for (int j = 0; j < NT; ++j) {  // relative to the running maximum
                    float* x = &s[j][i / 2][2 * (i & 1)];
                    const float2 y = fma2(make_float2(x[0], x[1]), mul2(ks2, fold[j]), fma2(base, qsum[j], neg_m[j]));
                    x[0] = y.x;
                    x[1] = y.y;
                }
            }
            // positions that some row does not see: their scores become -inf and their weights 0.
            // A scale that is not finite would still make NaN of a weight of 0 (`odd`).
            bool odd = false;
            if (__any_sync(kAll, here >= first_end)) {
                if constexpr (TOKENS) {
                    const float v = fabsf(__uint_as_float(reinterpret_cast<const uint2*>(tile + At::kScaleAt)[lane].y << 16));
                    const uint32_t mine = __float_as_uint(v < INFINITY ? v : 0.f);
                    const float all = __uint_as_float(__reduce_max_sync(kAll, mine));
                    if (all * wmul > kOver && all > 8.f * __uint_as_float(__reduce_max_sync(kAll, here < first_end ? mine : 0u))) {
                        const int e = end_past(__reduce_min_sync(kAll, here));  // of the rows that see something here
                        if (all > 8.f * __uint_as_float(__reduce_max_sync(kAll, here < e ? mine : 0u))) {
                            if (lane == 0) {
                                turn[0] = e;
                                turn[1] = upto;
                            }
                            if (here >= e) here = kNoPosition;
                            upto = j0 + 1;
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    at[i] = __shfl_sync(kAll, here, 8 * i + g);
                    if (TOKENS && at[i] == kNoPosition) vs[i] = vm[i] = 0.f;  // in another turn
                    odd |= !(fabsf(vs[i]) < INFINITY && fabsf(vm[i]) < INFINITY);
#pragma unroll
                    for (int j = 0; j < NT; ++j)
#pragma unroll
                        for (int c = 0; c < 2; ++c)
                            if (at[i] >= ends[j][c]) s[j][i / 2][2 * (i & 1) + c] = -INFINITY;
                }
                odd = __any_sync(kAll, odd);
            }
            // raise the running maxima where a score passes one by 2^kRaise (or is the first), and
            // r where a value scale leaves it behind
            float vw[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) vw[i] = vs[i] * wmul * sign;
            float2 high[NT];
            float most = -INFINITY;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                high[j].x = fmaxf(max3(s[j][0][0], s[j][0][2], s[j][1][0]), s[j][1][2]);
                high[j].y = fmaxf(max3(s[j][0][1], s[j][0][3], s[j][1][1]), s[j][1][3]);
                most = max3(most, high[j].x, high[j].y);
            }
            if (fresh || __any_sync(kAll, most > kRaise || fmaxf(max3(fabsf(vw[0]), fabsf(vw[1]), fabsf(vw[2])), fabsf(vw[3])) > kOver)) {
                float vtop = 1e-30f;
#pragma unroll
                for (int i = 0; i < 4; ++i) vtop = fmaxf(vtop, fabsf(vs[i]) < INFINITY ? fabsf(vs[i]) : 0.f);
                const uint32_t vbits = __reduce_max_sync(kAll, __float_as_uint(vtop));
                float change = 1.f;
                if (__uint_as_float(vbits) * wmul > kOver) {  // r = the power of two at or below vtop
                    const float to_mul = kTop / __uint_as_float(vbits & 0x7F800000u);
                    change = to_mul / wmul;
                    wmul = to_mul;
#pragma unroll
                    for (int i = 0; i < 4; ++i) vw[i] = vs[i] * (wmul * sign);
                }
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    float2 x = high[j];
#pragma unroll
                    for (int d = 4; d <= 16; d <<= 1) {
                        x.x = fmaxf(x.x, __shfl_xor_sync(kAll, x.x, d));
                        x.y = fmaxf(x.y, __shfl_xor_sync(kAll, x.y, d));
                    }
                    // a row's first score sets its maximum, up or down; nothing is summed yet
                    float2 by = make_float2(1.f, 1.f);
                    if (unseen >> (2 * j) & 1u) { if (x.x > -INFINITY) unseen &= ~(1u << (2 * j)); else x.x = 0.f; }
                    else { x.x = fmaxf(x.x, 0.f); by.x = exp2_fast(-x.x); }
                    if (unseen >> (2 * j + 1) & 1u) { if (x.y > -INFINITY) unseen &= ~(2u << (2 * j)); else x.y = 0.f; }
                    else { x.y = fmaxf(x.y, 0.f); by.y = exp2_fast(-x.y); }
                    const float2 down = make_float2(-x.x, -x.y);
                    neg_m[j] = add2(neg_m[j], down);
                    l[j] = mul2(l[j], by);
                    z[j] = mul2(z[j], by);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float* y = &s[j][i / 2][2 * (i & 1)];
                        y[0] += down.x;
                        y[1] += down.y;
                    }
                    const float2 all = mul2(by, both(change));
#pragma unroll
                    for (int mt = 0; mt < KS; ++mt) {
                        o[j][mt][0] *= all.x, o[j][mt][1] *= all.y;
                        o[j][mt][2] *= all.x, o[j][mt][3] *= all.y;
                    }
                    ones[j][0] *= all.x, ones[j][1] *= all.y;
                }
                fresh = __any_sync(kAll, unseen != 0u);
            }
            // weights p, their sums, and w as the second operand
            uint32_t wf[NT][2][2][NP];  // [row tile][16 positions][first or second 8][part]
            const auto weigh = [&](auto zeros) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 vw2 = both(vw[i]), vm2 = both(vm[i]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        const float* x = &s[j][i / 2][2 * (i & 1)];
                        const float2 e = make_float2(exp2_fast(x[0]), exp2_fast(x[1]));
                        l[j] = add2(l[j], e);
                        float2 w = mul2(e, vw2), zn = fma2(e, vm2, z[j]);
                        if (zeros.value) {
                            if (at[i] >= ends[j][0]) w.x = 0.f, zn.x = z[j].x;
                            if (at[i] >= ends[j][1]) w.y = 0.f, zn.y = z[j].y;
                        }
                        z[j] = zn;
                        uint32_t part[NP];
                        split_f16<NP>(w.x, w.y, part);
#pragma unroll
                        for (int n = 0; n < NP; ++n) wf[j][i / 2][i & 1][n] = transpose8x8(part[n]);
                    }
                }
            };
            if (!odd) weigh(std::false_type{});
            else weigh(std::true_type{});
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                // value words of positions 16 i + {2t, 2t + 1, 2t + 8, 2t + 9}, the lane's eighth
                uint32_t v[4][D / 64];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * i + 8 * (r >> 1) + 2 * t + (r & 1);
                    if constexpr (D == 128) {
                        const uint2 w = *reinterpret_cast<const uint2*>(tile + At::piece(row, 4 + (g >> 1)) + 8 * (g & 1));
                        v[r][0] = w.x, v[r][1] = w.y;
                    } else {
                        v[r][0] = *reinterpret_cast<const uint32_t*>(tile + At::piece(row, 2 + (g >> 2)) + 4 * (g & 3));
                    }
                    if (!CENTRE && (r & 1)) {  // complements at the odd positions
#pragma unroll
                        for (int w = 0; w < D / 64; ++w) v[r][w] = ~v[r][w];
                    }
                }
#pragma unroll
                for (int w = 0; w < D / 64; ++w) {
                    const uint32_t xl = __byte_perm(v[0][w], v[1][w], 0x5410), xh = __byte_perm(v[0][w], v[1][w], 0x7632);
                    const uint32_t yl = __byte_perm(v[2][w], v[3][w], 0x5410), yh = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
                    for (int nib = 0; nib < 4; ++nib) {
                        const int sh = nib >= 2 ? 8 : 0;
                        const uint32_t a0 = code_pair<CENTRE>(xl >> sh, nib), a1 = code_pair<CENTRE>(xh >> sh, nib);
                        const uint32_t a2 = code_pair<CENTRE>(yl >> sh, nib), a3 = code_pair<CENTRE>(yh >> sh, nib);
#pragma unroll
                        for (int j = 0; j < NT; ++j) {
                            float step[4] = {0.f, 0.f, 0.f, 0.f};
                            float(&sum)[4] = EXACT ? step : o[j][4 * w + nib];
#pragma unroll
                            for (int n = NP - 1; n >= 0; --n)
                                mma_f16(sum, a0, a1, a2, a3, wf[j][i][0][n], wf[j][i][1][n]);
                            if (EXACT) {
#pragma unroll
                                for (int c = 0; c < 4; ++c) o[j][4 * w + nib][c] += step[c];
                            }
                        }
                    }
                }
                if constexpr (!CENTRE) {  // even minus odd w, against ones
                    constexpr uint32_t ONE = 0x3C003C00u;
#pragma unroll
                    for (int j = 0; j < NT; ++j) mma_f16(ones[j], ONE, ONE, ONE, ONE, wf[j][i][0][0], wf[j][i][1][0]);
                }
            }
        }
        if constexpr (!TOKENS) break;
        __syncwarp();
        int past = turn[0];
        if (past == 0) break;
        // again the tile that was the last, for its next position, or on behind it
        int begin = past++;
        j0 -= STRIDE;
        if (begin >= min(j0 + kAttTile, last_end())) {
            j0 += STRIDE;
            begin = past = 0;
        }
        upto = past > 0 ? j0 + 1 : turn[1];
        copies_wait<0>();
        __syncwarp();
        if (lane == 0) turn[0] = past;
#pragma unroll
        for (int i = 0; i < kAttStages; ++i) ahead[i] = position_at(j0 + i * STRIDE + lane);
        at_far = position_at(j0 + kAttStages * STRIDE + lane);
        if (past > 0 && (ahead[0] < begin || ahead[0] >= past)) ahead[0] = -1;
#pragma unroll
        for (int i = 0; i < kAttStages; ++i) page[i] = page_of(ahead[i]);
#pragma unroll
        for (int i = 0; i + 1 < kAttStages; ++i) {
            const uint32_t entry = entry_of(ahead[i], page[i], pos[i]);
            issue(i, entry, is_run(entry));
        }
        at_ahead = ahead[kAttStages - 1];
        page_ahead = page[kAttStages - 1];
        slot = 0;
    }
    copies_wait<0>();
    __syncthreads();  // every warp is done with its ring

    // Join the warps: sums over the lanes of a row, then shared memory.  Output fragments stay as the
    // matrix unit leaves them, one float4 a lane, in shared memory and in the workspace: every access
    // is a run of 512 bytes.
    constexpr int NF = NT * KS;                          // fragments of a warp
    float4* sm_o = reinterpret_cast<float4*>(smem);      // [warps][NF][32]
    float4* sm_r = sm_o + WARPS * NF * 32;           // [warps][ROWS]: maximum, sum of p, of p (m + MID s)
    const float back = 1.f / wmul;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        float ls[2] = {l[j].x, l[j].y}, zs[2] = {z[j].x, z[j].y};
        const float ms[2] = {unseen >> (2 * j) & 1u ? kNone : -neg_m[j].x, unseen >> (2 * j) & 2u ? kNone : -neg_m[j].y};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
#pragma unroll
            for (int d = 4; d <= 16; d <<= 1) {
                ls[c] += __shfl_xor_sync(kAll, ls[c], d);
                zs[c] += __shfl_xor_sync(kAll, zs[c], d);
            }
            if (!CENTRE) zs[c] -= 7.5f * ones[j][c] * back;
            if (g == 0) sm_r[warp * ROWS + 8 * j + 2 * t + c] = make_float4(ms[c], ls[c], zs[c], 0.f);
        }
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
            const float f = mt & 1 ? kUnit * 0.0625f : kUnit;
            sm_o[(warp * NF + j * KS + mt) * 32 + lane] = make_float4(o[j][mt][0] * f * back, o[j][mt][1] * f * back,
                                                                      o[j][mt][2] * f * back, o[j][mt][3] * f * back);
        }
    }
    __syncthreads();
    // one warp joins the four fragments of a row tile j and code word w: they hold eight numbers in
    // a row of rows 2t and 2t + 1
    float4* sm_j = sm_r + WARPS * ROWS;              // the CTA's join, for its cluster: [NF][32]
    float2* sm_ml = reinterpret_cast<float2*>(sm_j + NF * 32);  // [ROWS]
    constexpr int ITEMS = NF / 4;
    const Emit<T, D> emit = {p, b, h, q0, picked, rg * ROWS, min(ROWS, p.rows - rg * ROWS), g, t};
    for (int item = warp; item < ITEMS; item += WARPS) {
        const int r = 8 * (item / (D / 64)) + 2 * t;
        float4 a0[WARPS], a1[WARPS];
        float top0 = kNone, top1 = kNone, sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            a0[w] = sm_r[w * ROWS + r];
            a1[w] = sm_r[w * ROWS + r + 1];
            top0 = fmaxf(top0, a0[w].x);
            top1 = fmaxf(top1, a1[w].x);
        }
        float4 acc[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[f] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f0 = exp2_fast(a0[w].x - top0), f1 = exp2_fast(a1[w].x - top1);
            sum0 += f0 * a0[w].y;
            sum1 += f1 * a1[w].y;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const float4 x = sm_o[(w * NF + item * 4 + f) * 32 + lane];
                acc[f].x += f0 * (x.x + a0[w].z), acc[f].y += f1 * (x.y + a1[w].z);
                acc[f].z += f0 * (x.z + a0[w].z), acc[f].w += f1 * (x.w + a1[w].z);
            }
        }
        if (splits == 1) {
            emit.four(item, acc, top0, sum0, top1, sum1);
            continue;
        }
        float4* to = p.cluster ? sm_j : p.ws_o + static_cast<int64_t>(blockIdx.x) * (NF * 32);
        float2* ml = p.cluster ? sm_ml : p.ws_ml + static_cast<int64_t>(blockIdx.x) * ROWS;
#pragma unroll
        for (int f = 0; f < 4; ++f) to[(item * 4 + f) * 32 + lane] = acc[f];
        if (g == 0 && item % (D / 64) == 0) {
            ml[r] = make_float2(top0, sum0);
            ml[r + 1] = make_float2(top1, sum1);
        }
    }
    if (!p.cluster) return;
    // every CTA of the cluster joins its share of the items from all of them
    cluster_sync_all();
    for (int item = warp * p.splits + split; item < ITEMS; item += WARPS * p.splits) {
        const int r = 8 * (item / (D / 64)) + 2 * t;
        float top0 = kNone, top1 = kNone, sum0 = 0.f, sum1 = 0.f;
        for (int c = 0; c < p.splits; ++c) {
            const uint4 ml = ld_cluster_v4(map_rank(sm_ml + r, c));  // rows r and r + 1
            top0 = fmaxf(top0, __uint_as_float(ml.x));
            top1 = fmaxf(top1, __uint_as_float(ml.z));
        }
        float4 acc[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) acc[f] = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = 0; c < p.splits; ++c) {
            const uint4 ml = ld_cluster_v4(map_rank(sm_ml + r, c));
            const float f0 = exp2_fast(__uint_as_float(ml.x) - top0), f1 = exp2_fast(__uint_as_float(ml.z) - top1);
            sum0 += f0 * __uint_as_float(ml.y);
            sum1 += f1 * __uint_as_float(ml.w);
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const uint4 x = ld_cluster_v4(map_rank(sm_j + (item * 4 + f) * 32 + lane, c));
                acc[f].x += f0 * __uint_as_float(x.x), acc[f].y += f1 * __uint_as_float(x.y);
                acc[f].z += f0 * __uint_as_float(x.z), acc[f].w += f1 * __uint_as_float(x.w);
            }
        }
        emit.four(item, acc, top0, sum0, top1, sum1);
    }
    cluster_sync_all();  // the others have read this CTA's share
}

// Joins the splits of a unit: a CTA takes FR fragments (four that belong together, or with few
// units one, so that more CTAs read), its warps take the splits in turn.  Only the splits that
// hold positions are read (the others wrote nothing); their order is fixed, so a call's result does
// not depend on timing.
template <typename T, int D, int NT, int FR>
__global__ void __launch_bounds__(1024) ds_attend_join_kernel(const AttendParams p) {
    constexpr int KS = D / 16, NF = NT * KS, ROWS = 8 * NT, PARTS = NF / FR;
    extern __shared__ __align__(128) unsigned char smem[];  // [warps][FR][32] float4, [warps][8] float
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    float4* sh_o = reinterpret_cast<float4*>(smem);
    float2* sh_l = reinterpret_cast<float2*>(sh_o + warps * FR * 32);
    pdl_launch_dependents();
    pdl_wait();
    const uint32_t unit = blockIdx.x / PARTS;
    const int first = static_cast<int>(blockIdx.x % PARTS) * FR;  // the CTA's first fragment
    const uint32_t uh = unit / static_cast<uint32_t>(p.row_groups);
    const int rg = static_cast<int>(unit - uh * p.row_groups);
    const int bq = static_cast<int>(uh / static_cast<uint32_t>(p.heads));
    const int h = static_cast<int>(uh - bq * p.heads);
    const bool picked = p.indices != nullptr;
    const int b = picked ? bq / p.Q : bq, q0 = picked ? bq % p.Q : 0;
    int64_t begin = static_cast<int64_t>(unit) * p.splits, apart = 1;  // its splits' CTAs
    int splits;
    if (p.fit > 0) {
        const int2 cut = p.ws_cut[unit];
        if (cut.y == 1) return;  // written by its only split
        begin = cut.x;
        apart = static_cast<int64_t>(p.heads) * p.row_groups;
        splits = cut.y;
    } else {
        const int count = picked ? p.K : max(min(p.lens[b], p.max_pos), 0);
        splits = max(1, min(p.splits, (count + p.chunk - 1) / p.chunk));
    }
    const int r = 8 * (first / KS) + 2 * t;
    const float4* ml = reinterpret_cast<const float4*>(p.ws_ml + begin * ROWS + r);
    const float4* part = p.ws_o + (begin * NF + first) * 32 + lane;
    float top0 = kNone, top1 = kNone, sum0 = 0.f, sum1 = 0.f;
#pragma unroll 4
    for (int s = g; s < splits; s += 8) {
        const float4 x = ml[s * apart * (ROWS / 2)];  // maximum and sum of rows r and r + 1
        top0 = fmaxf(top0, x.x);
        top1 = fmaxf(top1, x.z);
    }
#pragma unroll
    for (int d = 4; d <= 16; d <<= 1) {
        top0 = fmaxf(top0, __shfl_xor_sync(kAll, top0, d));
        top1 = fmaxf(top1, __shfl_xor_sync(kAll, top1, d));
    }
    float4 acc[FR];
#pragma unroll
    for (int f = 0; f < FR; ++f) acc[f] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = warp; s < splits; s += warps) {
        const float4 x = ml[s * apart * (ROWS / 2)];
        const float f0 = exp2_fast(x.x - top0), f1 = exp2_fast(x.z - top1);
        sum0 += f0 * x.y;
        sum1 += f1 * x.w;
#pragma unroll
        for (int f = 0; f < FR; ++f) {
            const float4 y = part[(s * apart * NF + f) * 32];
            acc[f].x += f0 * y.x, acc[f].y += f1 * y.y, acc[f].z += f0 * y.z, acc[f].w += f1 * y.w;
        }
    }
    if (warps > 1) {
#pragma unroll
        for (int f = 0; f < FR; ++f) sh_o[(warp * FR + f) * 32 + lane] = acc[f];
        if (g == 0) sh_l[warp * 4 + t] = make_float2(sum0, sum1);
        __syncthreads();
        if (warp != 0) return;
        for (int w = 1; w < warps; ++w) {
            const float2 x = sh_l[w * 4 + t];
            sum0 += x.x;
            sum1 += x.y;
#pragma unroll
            for (int f = 0; f < FR; ++f) {
                const float4 y = sh_o[(w * FR + f) * 32 + lane];
                acc[f].x += y.x, acc[f].y += y.y, acc[f].z += y.z, acc[f].w += y.w;
            }
        }
    }
    const Emit<T, D> emit = {p, b, h, q0, picked, rg * ROWS, min(ROWS, p.rows - rg * ROWS), g, t};
    if constexpr (FR == 4) emit.four(first / 4, acc, top0, sum0, top1, sum1);
    else emit.one(first, acc[0], top0, sum0, top1, sum1);
}

template <typename T, int D, int NT, int WARPS, bool TOKENS>
static ds_status attend(const AttendParams& p, int dev, int sms, int64_t units, cudaStream_t stream) {
    constexpr int PARTS = sizeof(T) == 2 ? 1 : 2;
    auto kern = ds_attend_kernel<T, D, NT, PARTS, PARTS, WARPS, TOKENS>;
    const size_t ring = static_cast<size_t>(WARPS) * kAttStages * TileAt<D>::kBytes + D / 16 * 32 * 8 * NT * PARTS + WARPS * 8;
    const size_t join = (static_cast<size_t>(WARPS) * (D + 4) + D + 2) * 8 * NT * sizeof(float);  // sm_o, sm_r, sm_j, sm_ml
    const size_t smem = ring > join ? ring : join;
    // the opt-in above 48 KB is a property of the kernel on a device: set once
    static std::atomic<bool> opted[64];
    if (smem > 48 * 1024 && !opted[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
            return DS_ERR_CUDA;
        opted[dev].store(true, std::memory_order_release);
    }
    const dim3 grid(static_cast<unsigned>(p.fit ? static_cast<int64_t>(p.fit) * p.heads * p.row_groups : units * p.splits));
    const ds_status st = launch_pdl(kern, grid, WARPS * 32, smem, p.cluster ? p.splits : 1, stream, p);
    if (st != DS_OK || p.splits == 1 || p.cluster) return st;
    const auto join_by = [&](auto kernel, int fr, int most) {
        int warps = 1;
        while (warps < most && 4 * warps < p.splits) warps <<= 1;
        const size_t bytes = warps > 1 ? static_cast<size_t>(warps) * (fr * 32 * 16 + 32) : 0;
        return launch_pdl(kernel, dim3(static_cast<unsigned>(units * (NT * D / 16) / fr)), warps * 32, bytes, 1, stream, p);
    };
    return units * (NT * D / 64) < 2 * sms ? join_by(ds_attend_join_kernel<T, D, NT, 1>, 1, 32)
                                           : join_by(ds_attend_join_kernel<T, D, NT, 4>, 4, 16);
}

template <typename T, int D>
static ds_status attend_rows(const AttendParams& p, int dev, int sms, int nt, int warps, int64_t units, cudaStream_t stream) {
    const auto by = [&](auto tiles, auto size) {
        constexpr int NT = decltype(tiles)::value, WARPS = decltype(size)::value;
        return p.Q > 1 && !p.indices ? attend<T, D, NT, WARPS, true>(p, dev, sms, units, stream)
                                     : attend<T, D, NT, WARPS, false>(p, dev, sms, units, stream);
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    using Warps = std::integral_constant<int, kAttWarps>;
    if (nt == 1) return warps == 1 ? by(One{}, One{}) : by(One{}, Warps{});
    return warps == 1 ? by(Two{}, One{}) : by(Two{}, Warps{});
}

// Query rows of a unit: the heads of a group, and for whole contexts the step's tokens as well.
static int64_t attend_unit_rows(int32_t tokens, int32_t q_heads, int32_t heads, bool picked) {
    return static_cast<int64_t>(q_heads / heads) * (picked ? 1 : tokens);
}
static int attend_row_tiles(int64_t rows) { return rows > 8 ? 2 : 1; }

// What a call's sizes have to be, whatever its pointers.
static ds_status attend_sizes(int32_t dtype, int64_t sequences, int32_t tokens, int32_t q_heads, int32_t D, int32_t heads,
                              int32_t page, int64_t table_width, bool picked, int32_t K) {
    if ((dtype != DS_BF16 && dtype != DS_FP32) || sequences < 0 || tokens < 1 || q_heads < 1 || heads < 1 ||
        q_heads % heads != 0 || page < 1 || table_width < 1 || K < 0)
        return DS_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || (page & (page - 1)) != 0) return DS_ERR_UNSUPPORTED;
    // positions and places of a list count in 31 bits
    constexpr int64_t kMost = int64_t(1) << 30;
    if (table_width > kMost / page || K > kMost) return DS_ERR_UNSUPPORTED;
    // units are blocks of a grid, 31 bits as well
    const int64_t rows = attend_unit_rows(tokens, q_heads, heads, picked), tile = 8 * attend_row_tiles(rows);
    if (rows > (1 << 20) || sequences > 0x7FFFFFFFLL / (picked ? tokens : 1) / heads / ((rows + tile - 1) / tile))
        return DS_ERR_UNSUPPORTED;
    return DS_OK;
}

// How a call is cut up, and the workspace that takes.
struct AttendPlan {
    int64_t units;
    int32_t rows, nt, row_groups, warps, splits, chunk, cluster, fit;
    size_t entries, bytes;  // rows of partial results; 0 bytes: no workspace
};

// span: the table's positions, or the list's length where `picked`
static ds_status attend_plan(int64_t sequences, int32_t tokens, int32_t q_heads, int32_t heads, int32_t D, bool picked,
                             int64_t span, int sms, AttendPlan& a) {
    a.rows = static_cast<int32_t>(attend_unit_rows(tokens, q_heads, heads, picked));
    a.nt = attend_row_tiles(a.rows);
    a.row_groups = (a.rows + 8 * a.nt - 1) / (8 * a.nt);
    a.units = sequences * (picked ? tokens : 1) * heads * a.row_groups;
    // Splits: as many as find a place on an SM at once, down to one tile a warp (4 contexts of 1M
    // positions and 16 rows: 131 us, twice as many 141, three times 150; 16 lists of 1024 positions,
    // 4 heads: 9.4, one more split 14.5).  Many units: up to four times as many, since their lengths
    // differ and the longest must not be left for the end (48 contexts of up to 8192 positions: once
    // 82.7 us, four times 77.6), but no shorter than 16 tiles a warp: a CTA costs 7 us beside its tiles
    // (304 units of 512 positions: one CTA each 11.4 us, four 30; 304 of 2048: 26.6, four each 47.6).
    // Units that many and that short are one warp's work each, since a CTA of four has little more than
    // its start and its join to do (2432 units of 512 positions: 53.6 us, with four warps 88.7; 608:
    // 20.9 and 24.5).  From 1024 positions on four warps win (1216 units: 33.0, one warp 35.5; 2432 of
    // up to 4096: 140 and 162), and so they do with few units (304 of 512: 11.4 and 15.0).
    a.warps = a.units >= 4LL * sms && span <= 4 * kAttWarps * kAttTile ? 1 : kAttWarps;
    const int64_t unit_tiles = a.warps * kAttTile;
    const int64_t places = static_cast<int64_t>(sms) * att_resident(a.nt, a.warps);
    const auto at_most = [&](int64_t n, int64_t least) {
        const int64_t most = (span + least - 1) / least;
        return n < most ? n : most;
    };
    int64_t splits = at_most(places / a.units > 1 ? places / a.units : 1, unit_tiles);
    if (2 * a.units >= places) {
        const int64_t many = at_most((4 * places + a.units - 1) / a.units, 16 * unit_tiles);
        if (splits < many) splits = many;
    }
    if (splits < 1) splits = 1;
    // Short contexts whose splits all run at once are split over a cluster, up to two tiles a warp.
    const bool few = a.units * splits <= places && span <= 2 * kAttCluster * unit_tiles;
    if (few && splits > kAttCluster) splits = kAttCluster;
    int64_t chunk = (span + splits - 1) / splits;
    chunk = (chunk + unit_tiles - 1) / unit_tiles * unit_tiles;
    if (chunk < unit_tiles) chunk = unit_tiles;
    splits = (span + chunk - 1) / chunk;
    if (splits < 1) splits = 1;
    a.splits = static_cast<int32_t>(splits);
    a.chunk = static_cast<int32_t>(chunk);
    if (a.units * splits > 0x7FFFFFFFLL || a.units * (a.nt * D / 16) > 0x7FFFFFFFLL) return DS_ERR_UNSUPPORTED;
    // Up to 8 splits of a list or of few short contexts are a cluster and join over its shared memory
    // (64 lists of 512 positions: 11.4 us, through the workspace 13.6; 4 contexts of 512, 8 heads: 7.4
    // and 8.4; one of 2048: 7.8 and 8.1).  Many contexts differ in length, and a cluster holds its
    // places until the longest split is done (48 of up to 8192 positions: 105 us, through the
    // workspace 81).
    a.cluster = (picked || few) && splits > 1 && splits <= kAttCluster;
    a.fit = 0;
    a.entries = a.bytes = 0;
    if (splits > 1 && !a.cluster) {
        // Few units with splits of at least four tiles a warp by the table's width: splits by the
        // lengths (16 contexts of up to 16384 positions, 8 heads: 40.0 us, by the width 59.7; 12 of up to
        // 4096: 16.3 and 17.9).  Finding them takes 1 to 1.5 us, which shorter splits or equal lengths
        // do not give back (16 of 16384: 62.0 and 60.6; one of 4096: 11.2 and 9.7).
        const int64_t per = a.units / sequences, steps = (span + unit_tiles - 1) / unit_tiles;
        int64_t partials = a.units * splits;
        if (!picked && 2 * a.units < places && span / splits >= 4 * unit_tiles && steps < (1 << 20)) {
            a.fit = static_cast<int32_t>(std::min(places / per, sequences * steps));
            partials = a.fit * per;
        }
        a.entries = static_cast<size_t>(partials) * 8 * a.nt;
        a.bytes = a.entries * (D + 2) * sizeof(float) + (a.fit ? a.units * sizeof(int2) : 0);
    }
    return DS_OK;
}

}  // namespace dsk

using namespace dsk;

extern "C" {

ds_status ds_cache_attention_ex(const void* q, int32_t dtype, int64_t sequences, int32_t tokens, int32_t q_heads,
                                int32_t D, int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride,
                                const void* cache, const void* scales, int64_t pages, int32_t heads, int32_t page,
                                const int32_t* table, int64_t table_width, int64_t table_stride, const int32_t* lens,
                                const int32_t* indices, int32_t K, float scale, void* out, float* out_lse,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    if (pages < 1 || table_stride < table_width || q_seq_stride < 0 || q_token_stride < 0 || q_head_stride < 0 || !isfinite(scale))
        return DS_ERR_INVALID_ARG;
    const ds_status sizes = attend_sizes(dtype, sequences, tokens, q_heads, D, heads, page, table_width, indices != nullptr, K);
    if (sizes != DS_OK) return sizes;
    if (pages > 0x7FFFFFFFLL || pages > 0xFFFFFFFELL / heads / page) return DS_ERR_UNSUPPORTED;  // 32 bits count entries
    if (sequences == 0) return DS_OK;
    if (!q || !cache || !scales || !table || !lens || !out || (K > 0 && !indices)) return DS_ERR_INVALID_ARG;
    const int es = dtype == DS_BF16 ? 2 : 4;
    if (!aligned16(cache) || reinterpret_cast<uintptr_t>(scales) % 8 || reinterpret_cast<uintptr_t>(q) % es ||
        !aligned16(out))
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
    p.scales = static_cast<const uint2*>(scales);
    p.table = table;
    p.table_stride = table_stride;
    p.lens = lens;
    p.indices = indices;
    p.out = out;
    p.lse = out_lse;
    p.max_pos = static_cast<int32_t>(table_width * page);
    p.span = indices ? K : p.max_pos;
    p.Q = tokens;
    p.K = K;
    p.heads = heads;
    p.group = q_heads / heads;
    while ((1 << p.page_log) < page) ++p.page_log;
    p.pages = static_cast<int32_t>(pages);
    p.scale = scale;
    // the stride of an extent of 1 is never used
    p.q_vec = aligned16(q) && (sequences == 1 || q_seq_stride * es % 16 == 0) &&
              (tokens == 1 || q_token_stride * es % 16 == 0) && (q_heads == 1 || q_head_stride * es % 16 == 0);
    AttendPlan a;
    const ds_status planned = attend_plan(sequences, tokens, q_heads, heads, D, indices != nullptr, p.span, info.sms, a);
    if (planned != DS_OK) return planned;
    p.rows = a.rows;
    p.row_groups = a.row_groups;
    p.splits = a.splits;
    p.chunk = a.chunk;
    p.cluster = a.cluster;
    p.fit = a.fit;
    p.sequences = static_cast<int32_t>(sequences);
    if (a.bytes > 0) {
        void* ws = workspace;
        if (!ws) {
            const ds_status st = library_workspace(dev, kWsAttend, a.bytes, stream, &ws);
            if (st != DS_OK) return st;
        } else if (workspace_bytes < a.bytes) {
            return DS_ERR_WORKSPACE;
        } else if (!aligned16(ws)) {
            return DS_ERR_ALIGNMENT;
        }
        p.ws_o = static_cast<float4*>(ws);
        p.ws_ml = reinterpret_cast<float2*>(static_cast<float*>(ws) + a.entries * D);
        p.ws_cut = reinterpret_cast<int2*>(p.ws_ml + a.entries);
    }
    if (dtype == DS_BF16)
        return D == 64 ? attend_rows<__nv_bfloat16, 64>(p, dev, info.sms, a.nt, a.warps, a.units, stream)
                       : attend_rows<__nv_bfloat16, 128>(p, dev, info.sms, a.nt, a.warps, a.units, stream);
    return D == 64 ? attend_rows<float, 64>(p, dev, info.sms, a.nt, a.warps, a.units, stream)
                   : attend_rows<float, 128>(p, dev, info.sms, a.nt, a.warps, a.units, stream);
}

ds_status ds_cache_attention(const void* q, int32_t dtype, int64_t sequences, int32_t tokens, int32_t q_heads,
                             int32_t D, int64_t q_seq_stride, int64_t q_token_stride, int64_t q_head_stride,
                             const void* cache, const void* scales, int64_t pages, int32_t heads, int32_t page,
                             const int32_t* table, int64_t table_width, int64_t table_stride, const int32_t* lens,
                             const int32_t* indices, int32_t K, float scale, void* out, float* out_lse,
                             cudaStream_t stream) {
    return ds_cache_attention_ex(q, dtype, sequences, tokens, q_heads, D, q_seq_stride, q_token_stride, q_head_stride,
                                 cache, scales, pages, heads, page, table, table_width, table_stride, lens, indices, K,
                                 scale, out, out_lse, nullptr, 0, stream);
}

ds_status ds_cache_attention_workspace_bytes(int32_t dtype, int64_t sequences, int32_t tokens, int32_t q_heads, int32_t D,
                                             int32_t heads, int32_t page, int64_t table_width, int32_t picked, int32_t K,
                                             size_t* bytes) {
    if (!bytes) return DS_ERR_INVALID_ARG;
    *bytes = 0;
    const ds_status sizes = attend_sizes(dtype, sequences, tokens, q_heads, D, heads, page, table_width, picked != 0, K);
    if (sizes != DS_OK || sequences == 0) return sizes;
    int dev = 0;
    DevInfo info;
    if (cudaGetDevice(&dev) != cudaSuccess || !dev_info(dev, info)) return DS_ERR_CUDA;
    AttendPlan a;
    const ds_status st = attend_plan(sequences, tokens, q_heads, heads, D, picked != 0, picked ? K : table_width * page, info.sms, a);
    if (st == DS_OK) *bytes = a.bytes;
    return st;
}

}  // extern "C"
